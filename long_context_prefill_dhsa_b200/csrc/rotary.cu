// Rotary positions of Q and K, with the append of K, V and positions to a cache.
//
// Pair i of a row at position p turns by a = p * inv_freq[i]. The angle is
// needed modulo one turn only, so it is kept as a fraction of a turn in 64-bit
// fixed point: F_i = inv_freq[i] / 2 pi mod 1, times 2^64, and p * F_i mod 2^64 is
// the fraction exactly as the integer product wraps (negative positions too).
// Its top 32 bits as a signed number are half-turns in [-1, 1), the argument of
// sincospif: at position 2^20 the angle is still good to fp32, where an fp32
// product would be off by 0.06 rad.
//
// HBM-bound: every row is read once and written once. A thread owns 16
// elements (32 bytes) of a token's row, eight of its pairs, in every head of
// its head group: it computes eight cosines and sines once and applies them
// to all those heads, so the trigonometry is shared by up to Hq + Hkv rows.
// Half layout: elements 8u .. 8u+7 and the same plus rotary_dim/2;
// interleaved: elements 16u .. 16u+15. Eight threads make a row, and a
// 16-byte access of the eight covers 128 contiguous bytes. Measured: 40 heads
// of 32768 tokens 108.5 us, 671 MB at 6.2 TB/s.
#include "cache.cuh"

namespace dhsa {
namespace {

constexpr int kRotThreads = 128;
constexpr int kUnits = kHeadDim / 16;   // threads per row
constexpr int kHeadsInFlight = 4;       // rows a thread has loaded at a time

struct RotaryParams {
  const __nv_bfloat16 *Q, *K, *V;
  __nv_bfloat16 *Qo, *Ko, *Vo;
  RowStrides qs, ks, vs, qos, kos, vos;
  const double* inv_freq;
  const int32_t *positions, *start, *n_new, *slots;
  int32_t* pos_out;
  int B, Hq, Hkv, T, cap;
  int rotary_dim;
  int rows;              // of a token: Q heads, K heads, V heads
  int heads_per_group;
  float sin_sign, factor;
  unsigned int* status;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

template <bool INTERLEAVED>
__device__ __forceinline__ void turn(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
  uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
  if (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = bf_lo(xw[i]), b = bf_hi(xw[i]);
      xw[i] = pack2(a * c[i] - b * s[i], a * s[i] + b * c[i]);
      const float d = bf_lo(yw[i]), e = bf_hi(yw[i]);
      yw[i] = pack2(d * c[4 + i] - e * s[4 + i], d * s[4 + i] + e * c[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = bf_lo(xw[i]), a1 = bf_hi(xw[i]), b0 = bf_lo(yw[i]), b1 = bf_hi(yw[i]);
      xw[i] = pack2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
      yw[i] = pack2(a0 * s[2 * i] + b0 * c[2 * i], a1 * s[2 * i + 1] + b1 * c[2 * i + 1]);
    }
  }
  x = make_uint4(xw[0], xw[1], xw[2], xw[3]);
  y = make_uint4(yw[0], yw[1], yw[2], yw[3]);
}

// STREAM: the outputs do not fit in L2
template <bool INTERLEAVED, bool STREAM>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryParams p) {
  const long long idx = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  const int u = (int)(idx % kUnits);
  const long long bt = idx / kUnits;
  if (bt >= (long long)p.B * p.T) return;
  const int b = (int)(bt / p.T), t = (int)(bt % p.T);
  if (p.n_new && t >= p.n_new[b]) return;

  const int pos = p.positions ? p.positions[bt] : (p.start ? p.start[b] : 0) + t;
  const int half = p.rotary_dim >> 1;
  const bool rotated = 16 * u < p.rotary_dim;
  // element offsets of the thread's two 16-byte words
  int e0 = 16 * u, e1 = 16 * u + 8;
  float c[8], s[8];
  if (rotated) {
    if (!INTERLEAVED) {
      e0 = 8 * u;
      e1 = half + 8 * u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      double f = p.inv_freq[8 * u + i] * 0.15915494309189533577;   // 1 / 2 pi
      f -= floor(f);
      const unsigned long long F = __double2ull_rn(f * 18446744073709551616.0);
      const unsigned long long a = F * (unsigned long long)(long long)pos;
      float sn, cs;
      // the top 32 bits, rounded to 24 by the conversion, as half-turns
      sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &sn, &cs);
      c[i] = cs * p.factor;
      s[i] = sn * p.factor * p.sin_sign;
    }
  }

  const int slot = (p.slots ? p.slots[b] : 0) + t;
  const bool writable = slot >= 0 && slot < p.cap;
  const int row0 = blockIdx.y * p.heads_per_group;
  const int row1 = min(row0 + p.heads_per_group, p.rows);
  if (!writable && row1 > p.Hq) raise_device_flag(p.status, DHSA_DEVFLAG_BAD_CACHE);

  for (int r0 = row0; r0 < row1; r0 += kHeadsInFlight) {
    uint4 x[kHeadsInFlight], y[kHeadsInFlight];
    __nv_bfloat16* dst[kHeadsInFlight];
#pragma unroll
    for (int k = 0; k < kHeadsInFlight; ++k) {
      const int r = r0 + k;
      const __nv_bfloat16* src = nullptr;
      dst[k] = nullptr;
      if (r < row1) {
        if (r < p.Hq) {
          if (p.Q) {
            src = p.Q + b * p.qs.b + r * p.qs.h + t * p.qs.r;
            dst[k] = p.Qo + b * p.qos.b + r * p.qos.h + t * p.qos.r;
          }
        } else if (r < p.Hq + p.Hkv) {
          const int h = r - p.Hq;
          if (p.K && writable) {
            src = p.K + b * p.ks.b + h * p.ks.h + t * p.ks.r;
            dst[k] = p.Ko + b * p.kos.b + h * p.kos.h + slot * p.kos.r;
            if (p.pos_out && u == 0) p.pos_out[((long long)b * p.Hkv + h) * p.cap + slot] = pos;
          }
        } else {
          const int h = r - p.Hq - p.Hkv;
          if (p.V && writable) {
            src = p.V + b * p.vs.b + h * p.vs.h + t * p.vs.r;
            dst[k] = p.Vo + b * p.vos.b + h * p.vos.h + slot * p.vos.r;
          }
        }
      }
      if (dst[k]) {
        x[k] = *reinterpret_cast<const uint4*>(src + e0);
        y[k] = *reinterpret_cast<const uint4*>(src + e1);
      }
    }
#pragma unroll
    for (int k = 0; k < kHeadsInFlight; ++k) {
      if (!dst[k]) continue;
      if (rotated && r0 + k < p.Hq + p.Hkv) turn<INTERLEAVED>(x[k], y[k], c, s);
      uint4 *d0 = reinterpret_cast<uint4*>(dst[k] + e0), *d1 = reinterpret_cast<uint4*>(dst[k] + e1);
      if (STREAM) {
        __stcs(d0, x[k]);
        __stcs(d1, y[k]);
      } else {
        *d0 = x[k];
        *d1 = y[k];
      }
    }
  }
}

}  // namespace

int launch_rotary(const void* Q, const RowStrides& qs, const void* K, const RowStrides& ks, const void* V,
                  const RowStrides& vs, int B, int Hq, int Hkv, int T, const double* inv_freq, int rotary_dim,
                  bool interleaved, bool transpose, float factor, const int32_t* positions, const int32_t* start,
                  const int32_t* n_new, void* Qo, void* Ko, const RowStrides& kos, void* Vo, const RowStrides& vos,
                  const int32_t* slots, int cap, int32_t* pos_out, unsigned int* status, cudaStream_t stream) {
  RotaryParams p;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.K = static_cast<const __nv_bfloat16*>(K);
  p.V = static_cast<const __nv_bfloat16*>(V);
  p.Qo = static_cast<__nv_bfloat16*>(Qo);
  p.Ko = static_cast<__nv_bfloat16*>(Ko);
  p.Vo = static_cast<__nv_bfloat16*>(Vo);
  p.qs = qs;
  p.ks = ks;
  p.vs = vs;
  p.qos = dense_strides(Hq, T);
  p.kos = kos;
  p.vos = vos;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.start = start;
  p.n_new = n_new;
  p.slots = slots;
  p.pos_out = pos_out;
  p.B = B;
  p.Hq = Q ? Hq : 0;
  p.Hkv = Hkv;
  p.T = T;
  p.cap = cap;
  p.rotary_dim = rotary_dim;
  p.sin_sign = transpose ? -1.f : 1.f;
  p.factor = factor;
  p.status = status;
  const int rows = p.rows = p.Hq + (V ? 2 : K ? 1 : 0) * Hkv;
  const long long blocks = ((long long)B * T * kUnits + kRotThreads - 1) / kRotThreads;
  // Few tokens: spread the heads over blocks until four blocks per SM exist.
  // More groups repeat the cosines and sines: 18 rows of 16K tokens take 29.7
  // us in 1024 blocks and 35.9 us in four times as many; the 40 rows of 32K
  // tokens are the same either way (113 us).
  int groups = 1;
  while (blocks * groups < 4 * 148 && groups < rows) groups *= 2;
  // Outputs beyond L2 (126 MB) are written past it: 108.5 against 112.9 us at
  // 335 MB; outputs that fit stay there for the next kernel (75 MB: 29.7
  // against 32.6 us even for this one).
  const bool past_l2 = (long long)B * T * rows * kHeadDim * 2 > 96ll << 20;
  p.heads_per_group = ceil_div(rows, groups);
  groups = ceil_div(rows, p.heads_per_group);
  const dim3 grid((unsigned)blocks, (unsigned)groups);
  auto* kernel = interleaved ? (past_l2 ? rotary_kernel<true, true> : rotary_kernel<true, false>)
                             : (past_l2 ? rotary_kernel<false, true> : rotary_kernel<false, false>);
  kernel<<<grid, kRotThreads, 0, stream>>>(p);
  return launch_status();
}

}  // namespace dhsa
