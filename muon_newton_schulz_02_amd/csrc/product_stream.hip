// C = P Q^T for few rows (16 of a group at a time): bound by reading Q, so nothing is
// staged.  A workgroup has 32 columns of C and all of k, each of its eight waves every
// eighth 128 bytes of it, so that the whole panel of Q (98 KB for 1536 of bfloat16) is
// asked for at once; the waves' sums meet in LDS.  MFMA fragments come straight from
// memory: lane 16 q + r holds 16 bytes of row r, at 16 q of every 64, and an instruction
// reads 16 rows x 64 bytes.  (Which k an element is does not matter, as long as both
// operands agree.)
//
// Two rows through 1536 x 6144 bfloat16 weights of one expert or two (19 or 38 MB) take
// 7.3 to 10.7 us with the launch, staged 32 x 128 tiles 13 to 16; 604 MB of 32 experts 81 to
// 99 us, at 6.1 to 7.4 TB/s, and 112.  (Tiles are for k that is not a multiple of 16 bytes, and
// for what the plan finds faster on them.)
#include "product_tile.h"

namespace muon {
namespace {

typedef float f32x4s __attribute__((ext_vector_type(4)));
constexpr int SNT = 512, SW = SNT / 64, SBN = 32;

template <bool F32, int EPI>
__global__ __launch_bounds__(SNT) void product_stream_kernel(const ProductArgs a, const int nt) {
  constexpr int ESZ = F32 ? 4 : 2, PARTS = F32 ? 3 : 1, U = F32 ? 2 : 3, ROWS = 16;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int wave_sum[SW];
  float* red = reinterpret_cast<float*>(smem);                 // [wave][512]
  int* pre = reinterpret_cast<int*>(smem + SW * 512 * 4);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int u0 = blockIdx.x / nt, j0 = (blockIdx.x - u0 * nt) * SBN, n = a.n - j0;
  int units = (a.rows + ROWS - 1) / ROWS;
  if (a.offsets) {
    group_sums<SNT>(a.groups, pre, wave_sum, tid, [&](int x) {
      int lo, end;
      group_range(a, x, lo, end);
      return (end - lo + ROWS - 1) / ROWS;
    });
    units = pre[a.groups];
  }
  // (once, but where groups overlap and have more rows than there are)
  for (int u = u0; u < units; u += gridDim.x / nt) {
    if (u != u0) __syncthreads();
    int g = 0, i0 = u * ROWS, hi = a.rows;
    if (a.offsets) {
      for (int end = a.groups; end - g > 1;) {
        const int mid = (g + end) / 2;
        if (pre[mid] <= u) g = mid;
        else end = mid;
      }
      int lo;
      group_range(a, g, lo, hi);
      i0 = lo + (u - pre[g]) * ROWS;
    }
    const int m = hi - i0;

    const int r16 = lane & 15, quarter = (lane >> 4) * 16;
    const char* q[2];
#pragma unroll
    for (int f = 0; f < 2; ++f)
      q[f] = reinterpret_cast<const char*>(a.q) + (g * a.es_q + int64_t(min(j0 + 16 * f + r16, a.n - 1)) * a.ld_q) * ESZ;
    const char* p = reinterpret_cast<const char*>(a.p) + int64_t(i0 + min(r16, m - 1)) * a.ld_p * ESZ;
    const int kb = a.k * ESZ, chunks = (kb + 127) / 128;
    f32x4s acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};

    // both halves of a 128-byte chunk; a piece past the end of k (a multiple of 16 bytes)
    // is zeros, read from the row's start
    auto load = [&](const char* row, int c, int h) {
      const int at = c * 128 + h * 64 + quarter;
      return *reinterpret_cast<gload16*>((gchar*)(row + (at < kb ? at : 0)));
    };
    auto clean = [&](u32x4 v, int c, int h) {
      const bool in = c * 128 + h * 64 + quarter < kb;
#pragma unroll
      for (int d = 0; d < 4; ++d) v[d] = in ? v[d] : 0u;
      return v;
    };
    for (int c0 = w; c0 < chunks; c0 += SW * U) {
      u32x4 fq[U][2][2], fp[U][2];
#pragma unroll
      for (int s = 0; s < U; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int f = 0; f < 2; ++f) fq[s][f][h] = load(q[f], c0 + s * SW, h);
          fp[s][h] = load(p, c0 + s * SW, h);
        }
#pragma unroll
      for (int s = 0; s < U; ++s) {
        const int c = c0 + s * SW;
        if (c >= chunks) continue;
        if (c == chunks - 1) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int f = 0; f < 2; ++f) fq[s][f][h] = clean(fq[s][f][h], c, h);
            fp[s][h] = clean(fp[s][h], c, h);
          }
        }
        auto mul = [&](f32x4s& d, const u32x4& x, const u32x4& y) {
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), d, 0, 0, 0);
        };
        if constexpr (!F32) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < 2; ++f) mul(acc[f], fq[s][f][h], fp[s][h]);
        } else {
          auto split8 = [&](const u32x4 (&v)[2], u32x4 (&o)[PARTS]) {
            u32x2 x[3], y[3];
            split4(v[0], x);
            split4(v[1], y);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) o[i] = u32x4{x[i][0], x[i][1], y[i][0], y[i][1]};
          };
          u32x4 sp[PARTS];
          split8(fp[s], sp);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            u32x4 sq[PARTS];
            split8(fq[s][f], sq);
            constexpr int QPART[6] = {0, 2, 1, 0, 1, 0}, PPART[6] = {2, 0, 1, 1, 0, 0};
#pragma unroll
            for (int x = 0; x < 6; ++x) mul(acc[f], sq[QPART[x] % PARTS], sp[PPART[x] % PARTS]);
          }
        }
      }
    }
    // lane's acc[f][e]: row lane % 16, column 16 f + 4 (lane / 16) + e
#pragma unroll
    for (int f = 0; f < 2; ++f) *reinterpret_cast<f32x4s*>(red + w * 512 + f * 256 + lane * 4) = acc[f];
    __syncthreads();
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < SW; ++x) v += red[x * 512 + tid];
    if constexpr (EPI == EPI_STORE) {
      const int row = (tid % 256) / 4 % 16, col = tid / 256 * 16 + tid % 256 / 64 * 4 + tid % 4;
      if (row < m && col < n) {
        const int64_t at = int64_t(i0 + row) * a.ld_out + j0 + col;
        if constexpr (F32) reinterpret_cast<float*>(a.out)[at] = v;
        else reinterpret_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(v);
      }
    } else {
      // a row's 32 columns to half a wave
      __syncthreads();
      red[tid] = v;
      __syncthreads();
      const SoftCap cap = soft_cap(a);
      const int row = tid / 32, col = tid % 32, i = i0 + row;
      const float l = red[col / 16 * 256 + (col % 16 / 4 * 16 + row) * 4 + col % 4];
      const bool in = row < m && col < n;
      const float y = !in ? -INFINITY : EPI == EPI_LSE_CAP ? capped_y<true>(l, cap) : l * LOG2E;
      float mx = y;
#pragma unroll
      for (int s = 1; s < 32; s *= 2) mx = fmaxf(mx, __shfl_xor(mx, s));
      float sum = in ? __builtin_amdgcn_exp2f(y - (mx == -INFINITY ? 0.f : mx)) : 0.f;
#pragma unroll
      for (int s = 1; s < 32; s *= 2) sum += __shfl_xor(sum, s);
      if (in) {
        if (j0 + col == target_of(a, i)) a.logit[i] = EPI == EPI_LSE_CAP ? y * LN2 : l;
        if (col == 0) a.stats[int64_t(i) * a.stat_tiles + j0 / SBN] = make_float2(mx, sum);
      }
    }
  }
}

template <bool F32>
hipError_t launch_rows(int epi, const ProductArgs& a, hipStream_t stream) {
  const int nt = (a.n + SBN - 1) / SBN;
  const int64_t grid = int64_t(nt) * (a.rows / 16 + std::min(a.groups, a.rows));
  const size_t lds = SW * 512 * 4 + (size_t(a.groups) + 1) * 4;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(SNT), lds, stream, a, nt);
    return hipGetLastError();
  };
  switch (epi) {
    case EPI_LSE: return go(product_stream_kernel<F32, EPI_LSE>);
    case EPI_LSE_CAP:
    case EPI_LSE_LARGE_CAP: return go(product_stream_kernel<F32, EPI_LSE_CAP>);
    default: return go(product_stream_kernel<F32, EPI_STORE>);
  }
}

}  // namespace

hipError_t launch_stream(int epi, const ProductArgs& a, hipStream_t stream) {
  return a.f32 ? launch_rows<true>(epi, a, stream) : launch_rows<false>(epi, a, stream);
}

}  // namespace muon
