// Products of the experts and of the head: the launcher, and the kernel for
// operands too narrow for 16-byte loads.
#include <algorithm>

#include "products_device.h"

namespace muon {
namespace {

constexpr int TS = NAIVE_TILE_N;      // rows and columns of a workgroup's tile at most
constexpr int SMALL_NT = 1024;

template <bool F32>
__device__ __forceinline__ float load_as(const void* p, int64_t i) {
  if constexpr (F32) return gmem(reinterpret_cast<const float*>(p))[i];
  else return bf16_bits_to_float(gmem(reinterpret_cast<const uint16_t*>(p))[i]);
}
__device__ __forceinline__ float load1(const void* p, int64_t i, int f32) {
  return f32 ? load_as<true>(p, i) : load_as<false>(p, i);
}

__device__ __forceinline__ void store1(void* p, int64_t i, float v, int f32) {
  if (f32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<uint16_t*>(p)[i] = float_to_bf16_bits(v);
}

// A workgroup of 2^(ti + tj + kl) threads: 2^ti x 2^tj elements of C, 2^kl threads for the
// terms of each.
struct SmallShape {
  int ti, tj, kl;
};

// A few columns or rows of C, or a few terms: operands with rows of less than 16 bytes.  The
// terms of an element go to as many threads as there are beside the elements, and are joined
// in LDS: what such products have is a long k (16384 rows of 4 and 1536 bfloat16: grad_W
// 147 us, and 5860 by a thread an element; grad_x of 4 from 1536 75 and 354).
template <int FORM, int EPI, bool F32>
__global__ __launch_bounds__(SMALL_NT) void product_small_kernel(const ProductArgs a, const SmallShape s) {
  __shared__ float red[SMALL_NT];
  constexpr bool tn = FORM == FORM_TN;
  // along k where k lies along memory, or along the columns
  const int tid = threadIdx.x, rest = tn ? tid : tid >> s.kl;
  const int kk = tn ? tid >> (s.ti + s.tj) : tid & ((1 << s.kl) - 1);
  const int tx = rest & ((1 << s.tj) - 1), ty = rest >> s.tj & ((1 << s.ti) - 1);
  const int nt = (a.n + (1 << s.tj) - 1) >> s.tj;
  const int per_group = ((tn ? a.m : a.rows) + (1 << s.ti) - 1) >> s.ti;
  const int64_t tiles = int64_t(a.groups) * per_group * nt;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int jt = int(t % nt), it = int(t / nt % per_group), g = int(t / nt / per_group);
    int lo, hi;
    group_range(a, g, lo, hi);
    const int m = tn ? a.m : hi - lo, k = tn ? hi - lo : a.k;
    const int i = (it << s.ti) + ty, j = (jt << s.tj) + tx;
    bool in = i < m && j < a.n;
    float c = 0.f;
    if (in) {
      const int64_t q0 = tn ? int64_t(lo) * a.ld_q : int64_t(g) * a.es_q;
#pragma unroll 8
      for (int x = kk; x < k; x += 1 << s.kl) {
        float pv = load_as<F32>(a.p, tn ? int64_t(lo + x) * a.ld_p + i : int64_t(lo + i) * a.ld_p + x);
        if (!F32 && FORM != FORM_NT && a.rest && a.target[lo + (tn ? x : i)] - a.col0 == (tn ? i : x)) pv += a.rest[lo + (tn ? x : i)];
        const float qv = load_as<F32>(a.q, FORM == FORM_NT ? q0 + int64_t(j) * a.ld_q + x : q0 + int64_t(x) * a.ld_q + j);
        c = __builtin_fmaf(pv, qv, c);
      }
    }
    if (s.kl > 0) {
      const int at = ty << s.tj | tx;
      __syncthreads();
      red[kk << (s.ti + s.tj) | at] = c;
      __syncthreads();
      if (kk == 0)
        for (int x = 1; x < 1 << s.kl; ++x) c += red[x << (s.ti + s.tj) | at];
      in = in && kk == 0;
    }
    if constexpr (EPI == EPI_STORE) {
      if (in) {
        int64_t row = tn ? i : lo + i;
        const int64_t base = tn ? int64_t(g) * a.es_out : 0;
        if (a.add) c += load1(a.add, base + row * a.ld_add + j, a.add_f32);
        if (a.map) row = a.map[row];
        store1(a.out, base + row * a.ld_out + j, c, a.out_f32);
      }
    } else if constexpr (EPI == EPI_LSE) {
      const SoftCap cap = soft_cap(a);
      const float y = !in ? -INFINITY : a.cap != 0.f ? capped_y<true>(c, cap_r(c, cap), cap) : c * LOG2E;
      float mx = y;
      for (int s = 1; s < TS; s *= 2) mx = fmaxf(mx, __shfl_xor(mx, s));
      float sum = in ? __builtin_amdgcn_exp2f(y - (mx == -INFINITY ? 0.f : mx)) : 0.f;
      for (int s = 1; s < TS; s *= 2) sum += __shfl_xor(sum, s);
      if (in) {
        if (j == target_of(a, i)) a.logit[i] = a.cap != 0.f ? y * LN2 : c;
        if (tx == 0) a.stats[int64_t(i) * a.stat_tiles + jt] = make_float2(mx, sum);
      }
    } else if (in) {
      const SoftCap cap = soft_cap(a);
      const float r = cap_r(c, cap), y = a.cap != 0.f ? capped_y<true>(c, r, cap) : c * LOG2E;
      float d = a.ga[i] * __builtin_amdgcn_exp2f(y - a.lse[i] * LOG2E);
      const bool target = j == target_of(a, i);
      if (target) d -= a.gb[i];
      if (a.cap != 0.f) d *= cap_slope(r);
      if (target && !F32) a.rest[i] = rest_of(d);
      store1(a.out, int64_t(i) * a.ld_out + j, d, a.out_f32);
    }
  }
}

template <int FORM, int EPI>
hipError_t launch_small(const ProductArgs& a, hipStream_t stream) {
  const int m = FORM == FORM_TN ? a.m : a.rows, k = FORM == FORM_TN ? a.rows : a.k;
  SmallShape s = {4, 4, 0};
  if (EPI == EPI_STORE) {
    s = {};
    while (s.ti < 4 && 1 << s.ti < m) ++s.ti;
    while (s.tj < 4 && 1 << s.tj < a.n) ++s.tj;
    // whole waves, and from there on 16 terms a thread at least
    while (1 << (s.ti + s.tj + s.kl) < SMALL_NT && (s.ti + s.tj + s.kl < 6 || 16 << s.kl < k)) ++s.kl;
  }
  const int64_t nt = (a.n + (1 << s.tj) - 1) >> s.tj, mt = (m + (1 << s.ti) - 1) >> s.ti;
  const int64_t tiles = int64_t(a.groups) * mt * nt;
  if (tiles == 0) return hipSuccess;
  const dim3 grid(unsigned(std::min<int64_t>(tiles, 1 << 16))), block(1u << (s.ti + s.tj + s.kl));
  if (a.f32) hipLaunchKernelGGL((product_small_kernel<FORM, EPI, true>), grid, block, 0, stream, a, s);
  else hipLaunchKernelGGL((product_small_kernel<FORM, EPI, false>), grid, block, 0, stream, a, s);
  return hipGetLastError();
}

}  // namespace

namespace {

constexpr int RT = 256;

// Adds the partial sums of what was cut along k (ProductPlan), in order, to the
// addend, and rounds.  A workgroup row (blockIdx.y) a group; four columns a thread.  Bound
// by memory: four parts of 8192 x 1536 (226 MB moved) 35 to 43 us.
template <int FORM>
__global__ __launch_bounds__(RT) void product_sum_kernel(const ProductArgs a) {
  extern __shared__ int pre[];
  __shared__ int wave_sum[RT / 64];
  const int g = blockIdx.y, tid = threadIdx.x;
  int lo, hi;
  group_range(a, g, lo, hi);
  int64_t slot = 0, rows_of, row0;
  int pieces, rows;
  if constexpr (FORM == FORM_TN) {
    if (hi - lo <= a.chunk) return;
    const int chunk = safe_chunk<RT>(a, pre, wave_sum, tid);
    pieces = pieces_of(hi - lo, chunk);
    if (pieces == 1) return;
    group_sums<RT>(a.groups, pre, wave_sum, tid, [&](int x) {
      int l, h;
      group_range(a, x, l, h);
      return pieces_of(h - l, chunk);
    });
    slot = 2 * int64_t(pre[g] - g);
    rows = a.m;
    rows_of = a.m;
    row0 = 0;
  } else {
    pieces = (a.k + a.chunk - 1) / a.chunk;
    rows = hi - lo;
    rows_of = a.rows;
    row0 = lo;
  }
  const int64_t ld = part_ld(a.n);
  const int quads = int(ld / 4);
  const int64_t base = FORM == FORM_TN ? g * a.es_out : 0;
  for (int64_t q = int64_t(blockIdx.x) * RT + tid; q < int64_t(rows) * quads; q += int64_t(gridDim.x) * RT) {
    const int64_t r = row0 + q / quads;
    const int c = int(q % quads) * 4, cnt = min(4, a.n - c);
    const float4* p = reinterpret_cast<const float4*>(a.part + (slot * rows_of + r) * ld + c);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t next = rows_of * (ld / 4);
    // eight loads at a time: few rows leave each thread a chain of them
    for (int i = 0; i < pieces; i += 8) {
      float4 v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i + e < pieces ? p[(i + e) * next] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s.x += v[e].x;
        s.y += v[e].y;
        s.z += v[e].z;
        s.w += v[e].w;
      }
    }
    float v[4] = {s.x, s.y, s.z, s.w};
    if (a.add) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < cnt) v[e] += load1(a.add, base + r * a.ld_add + c + e, a.add_f32);
    }
    const int64_t at = base + (a.map ? a.map[r] : r) * a.ld_out + c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < cnt) store1(a.out, at + e, v[e], a.out_f32);
  }
}

// The queue of TN's tiles (ProductPlan): groups by their number of rows, most first, by a
// bitonic sort.  One workgroup; 5 us for eight groups, 7 for 64: its barriers' latency.
constexpr int MAX_GROUPS = 2048;
__global__ __launch_bounds__(RT) void product_order_kernel(const ProductArgs a) {
  __shared__ uint64_t key[MAX_GROUPS];
  __shared__ int pre[MAX_GROUPS + 1], rows[MAX_GROUPS];
  __shared__ int wave_sum[RT / 64];
  const int tid = threadIdx.x;
  int32_t* pre_out = a.queue + QUEUE_PRE;
  int32_t* order_out = pre_out + a.groups + 1;
  int32_t* slot_out = order_out + a.groups;
  for (int g = tid; g < a.groups; g += RT) {
    int lo, hi;
    group_range(a, g, lo, hi);
    rows[g] = hi - lo;
  }
  // (a thread reads the rows that it wrote)
  group_sums<RT>(a.groups, pre, wave_sum, tid, [&](int g) { return rows[g]; });
  const int chunk = pre[a.groups] <= a.rows ? a.chunk : 1 << 30;      // as safe_chunk
  __syncthreads();
  if (tid < QUEUE_XCD) a.queue[tid * QUEUE_STEP] = 0;
  if (tid == 0) a.queue[QUEUE_CHUNK] = chunk;
  group_sums<RT>(a.groups, pre, wave_sum, tid, [&](int g) { return pieces_of(rows[g], chunk); });
  int size = 1;
  while (size < a.groups) size *= 2;
  for (int g = tid; g < size; g += RT) {
    if (g < a.groups) slot_out[g] = 2 * (pre[g] - g);
    key[g] = g < a.groups ? uint64_t(uint32_t(~rows[g])) << 32 | uint32_t(g) : ~uint64_t(0);
  }
  __syncthreads();
  for (int run = 2; run <= size; run *= 2) {
    for (int apart = run / 2; apart > 0; apart /= 2) {
      for (int i = tid; i < size / 2; i += RT) {
        const int x = i / apart * 2 * apart + i % apart, y = x + apart;
        const uint64_t kx = key[x], ky = key[y];
        if ((kx > ky) == ((x & run) == 0)) {
          key[x] = ky;
          key[y] = kx;
        }
      }
      __syncthreads();
    }
  }
  group_sums<RT>(a.groups, pre, wave_sum, tid, [&](int i) { return pieces_of(int(~uint32_t(key[i] >> 32)), chunk); });
  for (int i = tid; i < a.groups; i += RT) {
    order_out[i] = int(uint32_t(key[i]));
    pre_out[i] = pre[i];
  }
  if (tid == 0) pre_out[a.groups] = pre[a.groups];
}

template <int FORM>
hipError_t launch_sum(const ProductArgs& a, int cus, hipStream_t stream) {
  const int64_t rows = FORM == FORM_TN ? a.m : std::max(1, a.rows / a.groups);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((rows * part_ld(a.n) / 4 + RT - 1) / RT, cus * 16 / a.groups + 1));
  hipLaunchKernelGGL((product_sum_kernel<FORM>), dim3(unsigned(blocks), unsigned(a.groups)), dim3(RT),
                     (size_t(a.groups) + 1) * 4, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product(int form, int epi, const ProductArgs& args, int cus, char* ws, hipStream_t stream) {
  const ProductPlan plan = product_plan(form, epi, args, cus);
  ProductArgs a = args;
  if (plan.shape != SHAPE_NAIVE) {
    a.chunk = plan.chunk;
    a.queue = plan.queue ? reinterpret_cast<int32_t*>(ws) : nullptr;
    a.part = reinterpret_cast<float*>(ws + plan.queue);
    const int kind = product_epilogue(epi, a);
    if (plan.shape == SHAPE_STREAM) return launch_stream(kind, a, stream);
    if (plan.queue) {
      hipLaunchKernelGGL(product_order_kernel, dim3(1), dim3(RT), 0, stream, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipError_t e = form == FORM_NT   ? launch_nt(plan.shape, kind, a, cus, stream)
                   : form == FORM_NN ? launch_nn(plan.shape, kind, a, cus, stream) : launch_tn(plan.shape, kind, a, cus, stream);
    if (e == hipSuccess && plan.bytes > plan.queue)
      e = form == FORM_TN ? launch_sum<FORM_TN>(a, cus, stream) : launch_sum<FORM_NT>(a, cus, stream);
    return e;
  }
  if (epi == EPI_LSE) return launch_small<FORM_NT, EPI_LSE>(a, stream);
  if (epi == EPI_DZ) return launch_small<FORM_NT, EPI_DZ>(a, stream);
  switch (form) {
    case FORM_NT: return launch_small<FORM_NT, EPI_STORE>(a, stream);
    case FORM_NN: return launch_small<FORM_NN, EPI_STORE>(a, stream);
    default: return launch_small<FORM_TN, EPI_STORE>(a, stream);
  }
}

}  // namespace muon
