// Kernels of the head's loss beside its products: the packing of the rows that
// have a target, and the loss from the tiles' maxima and sums.
#include <algorithm>

#include "products_device.h"

namespace muon {
namespace {

constexpr int NT = 256;

template <class A>
__device__ __forceinline__ bool has_target(const A& a, int64_t t) {
  return t != a.ignore_index && t >= 0 && t < a.vocab;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));   // 16 bytes at any element

// A row of n elements by a wave, 16 bytes a lane; src null: zeros.
template <class T>
__device__ __forceinline__ void copy_row(T* dst, const T* src, int n, int lane) {
  constexpr int V = 16 / sizeof(T);
  const int whole = n / V;
  for (int c = lane; c < whole; c += 64)
    *gmem(reinterpret_cast<u32x4_any*>(dst + c * V)) =
        src ? *gmem(reinterpret_cast<const u32x4_any*>(src + c * V)) : u32x4_any{0, 0, 0, 0};
  for (int c = whole * V + lane; c < n; c += 64) dst[c] = src ? src[c] : T(0);
}

// Each workgroup packs `chunk` rows: it counts the rows with a target before
// them by itself (8 bytes a row, read from L2), which saves a launch and a wait;
// the chunks are cut so that about a thousand workgroups at most do it.  The copy of x gives
// the products rows at 16-byte boundaries, and takes ignored rows out of them:
// their work, and whatever their x holds.  Bound by memory and the wait for the count: 8192
// rows of 1536 bfloat16 (50 MB read and written) 13 to 16 us.
template <class T>
__global__ __launch_bounds__(NT) void head_rows_kernel(const HeadRows a) {
  __shared__ int wave_sum[NT / 64];
  __shared__ int place[NT];   // where a row of this step goes, or -1
  __shared__ int start;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r0 = blockIdx.x * a.chunk, r1 = min(r0 + a.chunk, a.rows);
  int before = 0;
#pragma unroll 8
  for (int r = tid; r < r0; r += NT) before += has_target(a, a.targets[r]) ? 1 : 0;
  for (int s = 1; s < 64; s *= 2) before += __shfl_xor(before, s);
  if (lane == 0) wave_sum[wave] = before;
  __syncthreads();
  if (tid == 0) {
    int s = 0;
    for (int w = 0; w < NT / 64; ++w) s += wave_sum[w];
    start = s;
  }
  __syncthreads();
  int pos0 = start;
  for (int b = r0; b < r1; b += NT) {
    const int r = b + tid;
    const int64_t t = r < r1 ? a.targets[r] : a.ignore_index;
    const bool seen = r < r1 && has_target(a, t);
    const uint64_t votes = __ballot(seen);
    __syncthreads();
    if (lane == 0) wave_sum[wave] = __popcll(votes);
    __syncthreads();
    int at = pos0 + __popcll(votes & ((uint64_t(1) << lane) - 1)), all = 0;
    for (int w = 0; w < NT / 64; ++w) {
      if (w < wave) at += wave_sum[w];
      all += wave_sum[w];
    }
    pos0 += all;
    if (seen) {
      a.row[at] = r;
      a.target[at] = int(t);
      if (a.lse_in) {
        const float g = a.grad_loss[r], h = a.grad_lse ? a.grad_lse[r] : 0.f;
        a.lse_c[at] = a.lse_in[r];
        a.ga[at] = g + h;
        a.gb[at] = g;
      }
    } else if (r < r1 && a.loss) {
      const float v = t == a.ignore_index ? 0.f : __builtin_nanf("");
      a.loss[r] = v;
      a.lse_out[r] = v;
    }
    place[tid] = seen ? at : -1;
    __syncthreads();
    // the rows of x, a wave each
    const int rows = min(NT, r1 - b);
    const T* x = reinterpret_cast<const T*>(a.x);
    T* xc = reinterpret_cast<T*>(a.xc);
    T* gx = reinterpret_cast<T*>(a.grad_x);
    for (int w = wave; w < rows; w += NT / 64) {
      const int p = place[w];
      if (p >= 0) {
        copy_row(xc + int64_t(p) * a.ld_xc, x + int64_t(b + w) * a.ld_x, a.dim, lane);
      } else if (gx) {
        copy_row(gx + int64_t(b + w) * a.ld_grad_x, static_cast<const T*>(nullptr), a.dim, lane);
      }
    }
  }
  if (r1 == a.rows && tid == 0) {
    a.offsets[0] = 0;
    a.offsets[1] = pos0;
  }
}

// W waves a row: the maximum over the tiles, the sums brought to it.  Four where there
// are few rows, whose thousand tiles would be a chain of 16 loads for one (one row of 32768
// columns 4.0 us; 8192 rows of 128 tiles, a wave each, 5.4).
template <int W>
__global__ __launch_bounds__(NT) void head_finish_kernel(const HeadFinish a) {
  __shared__ float2 part[NT / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = blockIdx.x * (NT / 64 / W) + wave / W;
  const bool row = i < (a.targets ? a.rows : min(a.offsets[1], a.rows));
  const bool ignored = row && a.targets && !has_target(a, a.targets[i]);
  float m = -INFINITY, sum = 0.f;
  auto join = [&](float om, float os) {
    const float n = fmaxf(m, om), f = n == -INFINITY ? 0.f : n;
    sum = sum * __builtin_amdgcn_exp2f(m - f) + os * __builtin_amdgcn_exp2f(om - f);
    m = n;
  };
  if (row && !ignored) {
    const float2* s = a.stats + int64_t(i) * a.tiles;
    for (int t = lane + 64 * (wave % W); t < a.tiles; t += 64 * W) join(s[t].x, s[t].y);
  }
  for (int d = 1; d < 64; d *= 2) join(__shfl_xor(m, d), __shfl_xor(sum, d));
  if constexpr (W > 1) {
    if (lane == 0) part[wave] = make_float2(m, sum);
    __syncthreads();
    m = -INFINITY;
    sum = 0.f;
    for (int w = 0; w < W; ++w) join(part[wave / W * W + w].x, part[wave / W * W + w].y);
  }
  if (!row || lane != 0 || wave % W != 0) return;
  const int r = a.targets ? i : a.row[i];
  if (ignored) {
    a.loss[r] = a.lse[r] = a.targets[i] == a.ignore_index ? 0.f : __builtin_nanf("");
    return;
  }
  const float lse = __builtin_fmaf(m == -INFINITY ? 0.f : m, LN2, logf(sum));
  a.lse[r] = lse;
  a.loss[r] = lse - a.logit[i];
}

}  // namespace

hipError_t launch_head_rows(const HeadRows& a, hipStream_t stream) {
  const unsigned grid = unsigned((a.rows + a.chunk - 1) / a.chunk);
  if (a.f32) hipLaunchKernelGGL((head_rows_kernel<float>), dim3(grid), dim3(NT), 0, stream, a);
  else hipLaunchKernelGGL((head_rows_kernel<uint16_t>), dim3(grid), dim3(NT), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_head_finish(const HeadFinish& a, hipStream_t stream) {
  const int waves = a.rows <= 1024 ? 4 : 1, per = NT / 64 / waves;
  const dim3 grid(unsigned((a.rows + per - 1) / per));
  if (waves == 4) hipLaunchKernelGGL(head_finish_kernel<4>, grid, dim3(NT), 0, stream, a);
  else hipLaunchKernelGGL(head_finish_kernel<1>, grid, dim3(NT), 0, stream, a);
  return hipGetLastError();
}

}  // namespace muon
