// Products of the experts and of the head: the launcher, and the kernel for
// operands too small for 16-byte loads.
#include <algorithm>

#include "products_device.h"

namespace muon {
namespace {

constexpr int TS = 16;  // a workgroup's tile: 16 x 16, one element a thread

__device__ __forceinline__ float load1(const void* p, int64_t i, int f32) {
  return f32 ? reinterpret_cast<const float*>(p)[i] : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ void store1(void* p, int64_t i, float v, int f32) {
  if (f32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<uint16_t*>(p)[i] = float_to_bf16_bits(v);
}

// One element of C a thread, straight from the definition.
template <int FORM, int EPI>
__global__ __launch_bounds__(TS * TS) void product_small_kernel(const ProductArgs a) {
  const int tx = threadIdx.x % TS, ty = threadIdx.x / TS;
  const int nt = (a.n + TS - 1) / TS;
  const bool tn = FORM == FORM_TN;
  const int per_group = tn ? (a.m + TS - 1) / TS : (a.rows + TS - 1) / TS;
  const int64_t tiles = int64_t(a.groups) * per_group * nt;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int jt = int(t % nt), it = int(t / nt % per_group), g = int(t / nt / per_group);
    int lo, hi;
    group_range(a, g, lo, hi);
    const int m = tn ? a.m : hi - lo, k = tn ? hi - lo : a.k;
    const int i = it * TS + ty, j = jt * TS + tx;
    const bool in = i < m && j < a.n;
    float c = 0.f;
    if (in) {
      const int64_t q0 = tn ? int64_t(lo) * a.ld_q : int64_t(g) * a.es_q;
      for (int x = 0; x < k; ++x) {
        const float pv = tn ? load1(a.p, int64_t(lo + x) * a.ld_p + i, a.f32) : load1(a.p, int64_t(lo + i) * a.ld_p + x, a.f32);
        const float qv = FORM == FORM_NT ? load1(a.q, q0 + int64_t(j) * a.ld_q + x, a.f32)
                                         : load1(a.q, q0 + int64_t(x) * a.ld_q + j, a.f32);
        c += pv * qv;
      }
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
      const float z = in ? soft_capped(c, a.cap, a.inv_cap) : -INFINITY;
      float mx = z;
      for (int s = 1; s < TS; s *= 2) mx = fmaxf(mx, __shfl_xor(mx, s));
      float sum = in ? __expf(z - (mx == -INFINITY ? 0.f : mx)) : 0.f;
      for (int s = 1; s < TS; s *= 2) sum += __shfl_xor(sum, s);
      if (in) {
        if (j == a.target[i]) a.logit[i] = z;
        if (tx == 0) a.stats[int64_t(i) * a.stat_tiles + jt] = make_float2(mx, sum);
      }
    } else if (in) {
      const float z = soft_capped(c, a.cap, a.inv_cap);
      const float d = logit_gradient(a, z, a.col0 + j, a.target[i], a.lse[i], a.ga[i], a.gb[i]);
      store1(a.out, int64_t(i) * a.ld_out + j, d, a.out_f32);
    }
  }
}

template <int FORM, int EPI>
hipError_t launch_small(const ProductArgs& a, hipStream_t stream) {
  const int64_t nt = (a.n + TS - 1) / TS, mt = ((FORM == FORM_TN ? a.m : a.rows) + TS - 1) / TS;
  const int64_t tiles = int64_t(a.groups) * mt * nt;
  if (tiles == 0) return hipSuccess;
  hipLaunchKernelGGL((product_small_kernel<FORM, EPI>), dim3(unsigned(std::min<int64_t>(tiles, 1 << 16))),
                     dim3(TS * TS), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

namespace {

int product_shape(int form, const ProductArgs& a, int cus) {
  const int64_t esz = a.f32 ? 4 : 2;
  // 16-byte loads (product_tile.h)
  if (a.p_elems * esz < 16 || a.q_elems * esz < 16 || (form == FORM_TN && a.ld_p * esz < 16) ||
      (form != FORM_NT && a.ld_q * esz < 16))
    return SHAPE_NAIVE;
  const int64_t rows = form == FORM_TN ? a.m : a.rows / a.groups;       // of a group, on average
  if (form != FORM_TN && rows <= 32) return SHAPE_SMALL;
  const int64_t groups = form == FORM_TN ? a.groups : std::max<int64_t>(1, std::min<int64_t>(a.groups, a.rows / 256));
  const int64_t large = groups * ((rows + 255) / 256) * ((a.n + 255) / 256);
  return large >= cus ? SHAPE_LARGE : SHAPE_MEDIUM;
}

}  // namespace

int32_t product_tile_n(int form, const ProductArgs& a, int cus) {
  switch (product_shape(form, a, cus)) {
    case SHAPE_NAIVE: return TS;
    case SHAPE_LARGE: return a.f32 ? 128 : 256;
    default: return 128;
  }
}

hipError_t launch_product(int form, int epi, const ProductArgs& a, int cus, hipStream_t stream) {
  const int shape = product_shape(form, a, cus);
  if (shape != SHAPE_NAIVE)
    return form == FORM_NT ? launch_nt(shape, epi, a, cus, stream)
           : form == FORM_NN ? launch_nn(shape, a, cus, stream) : launch_tn(shape, a, cus, stream);
  if (epi == EPI_LSE) return launch_small<FORM_NT, EPI_LSE>(a, stream);
  if (epi == EPI_DZ) return launch_small<FORM_NT, EPI_DZ>(a, stream);
  switch (form) {
    case FORM_NT: return launch_small<FORM_NT, EPI_STORE>(a, stream);
    case FORM_NN: return launch_small<FORM_NN, EPI_STORE>(a, stream);
    default: return launch_small<FORM_TN, EPI_STORE>(a, stream);
  }
}

}  // namespace muon
