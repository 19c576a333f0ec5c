// moe_swiglu's and moe_swiglu_backward's kernels and the rule that shapes their workgroups, cut from csrc/swiglu.hip,
// on the host: the threads of a workgroup run one after another, so that a thread which reads what another one has
// written in place, or a chunk that two threads own, shows every time.
#include "shim.hpp"

namespace moe {
enum { kNear = 0, kReadOnce = 1, kThrough = 2 };
static float* g_out;        // the stores that are counted begin here
static std::vector<int> g_stores;

template <int DT>
struct Chunk {  // fp32 only
  float v[8];
  template <bool NT = false>
  void load(const void* row, int64_t at) { std::memcpy(v, (const float*)row + at, sizeof v); }
  void get(float* f) const { std::memcpy(f, v, sizeof v); }
};
template <int DT, bool NT = false>
void st8(void* row, int64_t at, const float* v) {
  float* o = (float*)row + at;
  std::memcpy(o, v, 8 * sizeof *v);
  const int64_t chunk = (o - g_out) / 8;
  if (chunk >= 0 && chunk < (int64_t)g_stores.size()) ++g_stores[chunk];
}
// (8-bit outputs are not built here)
struct Coding {
  float scale;
  void operator()(float*) const {}
};
inline float run_max(float v, int) { return v; }
inline Coding coding_of(float, float, bool) { return {1.f}; }
inline unsigned grid_of(int64_t units) { return (unsigned)(units < (1 << 20) ? units : 1 << 20); }
}  // namespace moe

#define __builtin_amdgcn_exp2f exp2f
#define __builtin_amdgcn_rcpf(x) (1.f / (x))
#include "swiglu_kernels.inc"

using namespace moe;

template <typename F>
static void one_after_another(unsigned grid, unsigned block, F f) {
  blockDim = {(int)block, 1, 1};
  gridDim = {(int)grid, 1, 1};
  for (int b = 0; b < (int)grid; ++b)
    for (int t = 0; t < (int)block; ++t) {
      blockIdx = {b, 0, 0};
      threadIdx = {t, 0, 0};
      f();
    }
}

static int wrong(const char* what, int I, unsigned block, const SwigluJob& j) {
  std::printf("%s: I %d, workgroups of %u threads, %d to a row\n", what, I, block, j.tpr);
  return 1;
}

static int check(int I, bool full) {
  SwigluJob j = {};
  j.I = I;
  j.n = 1;
  unsigned grid, block;
  swiglu_shape(j, grid, block);
  const int n = j.n = j.many + 1;
  swiglu_shape(j, grid, block);
  if (block > (unsigned)kSwigluT || block % 64 || j.tpr % 16 || (int)block < j.tpr * j.many || (int64_t)grid * j.many < n)
    return wrong("shape", I, block, j);
  std::vector<float> gu((size_t)n * 2 * I), dh((size_t)n * I), h(dh.size()), out(gu.size());
  for (size_t i = 0; i < gu.size(); ++i) gu[i] = (float)((int)(i * 7919 % 257) - 128) / 32.f;
  for (size_t i = 0; i < dh.size(); ++i) dh[i] = (float)((int)(i * 6007 % 129) - 64) / 16.f;
  j.gu_pitch = j.dgu_pitch = 2 * I;
  j.dh_pitch = j.h_pitch = I;
  j.gu = gu.data();
  j.dh = dh.data();
  // forward: every chunk stored once
  j.h = g_out = h.data();
  g_stores.assign(h.size() / 8, 0);
  one_after_another(grid, block, [&] { swiglu_kernel<MOE_F32, MOE_F32, kNear>(j); });
  for (int s : g_stores)
    if (s != 1) return wrong("forward", I, block, j);
  // the gradient: every chunk stored once, in place too, with the same results
  std::vector<float> again(h.size());
  j.h = again.data();
  j.dgu = g_out = out.data();
  g_stores.assign(out.size() / 8, 0);
  one_after_another(grid, block, [&] { swiglu_backward_kernel<MOE_F32, kNear>(j); });
  for (int s : g_stores)
    if (s != 1) return wrong("gradient", I, block, j);
  if (!full) return 0;
  if (again != h) return wrong("rows again", I, block, j);
  std::fill(again.begin(), again.end(), 0.f);
  j.dgu = g_out = gu.data();
  g_stores.assign(gu.size() / 8, 0);
  one_after_another(grid, block, [&] { swiglu_backward_kernel<MOE_F32, kNear>(j); });
  for (int s : g_stores)
    if (s != 1) return wrong("gradient in place", I, block, j);
  if (gu != out) return wrong("values in place", I, block, j);
  if (again != h) return wrong("rows again in place", I, block, j);
  return 0;
}

int main(int argc, char**) {
  int bad = 0;
  for (int I = 8; I <= 32768; I += 8) bad += check(I, argc > 1 || I % 424 == 0 || (I > 4096 && I < 6000));
  std::printf("%d of 4096 row lengths wrong\n", bad);
  return bad != 0;
}
