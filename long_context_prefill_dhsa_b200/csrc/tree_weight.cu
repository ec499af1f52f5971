// Attention weight of each cache slot: weight_out = weight + sum over the rows
// (query heads of the group x drafted tokens) of p = exp(scale (s - M)) / l,
// with each row's largest score M and denominator l from the attention.
//
// The scores are computed again, transposed: S^T = K Q^T puts the slots on the
// tensor core's M side, so that a thread owns a TMEM lane, one slot, and adds
// its rows' p with no exchange between threads. The rows' statistics enter in
// the tensor core too: two more steps of 16 columns, ones against -M and ones
// against -log2(l) / scale (each as three bf16 parts), leave the exponent in
// TMEM, so the epilogue reads nothing but its column. (Read from shared memory
// per pair of rows instead, they took a quarter of the kernel's time.) K is read once more (256
// bytes per slot); up to about 180 rows that read is the bound, above them
// the exponentials (16 per cycle and SM). Measured: 256 rows of 8 heads over
// 131008 slots 93 us, 2.9e12 exponentials a second, 64% of what the units can do.
//
// Warp 0 streams the K tiles, warp 1 issues the MMAs into two S^T buffers of
// 256 columns; eight warps take the even and eight the odd tiles, four for each
// half of the columns.
// More than 256 rows walk the same keys again and add to weight_out.
// Waits are bounded as in tree_attn.cu.
#include <type_traits>

#include "tree.cuh"

namespace dhsa {
namespace {

constexpr int kThreads = 640;
constexpr int BN = 128;                      // slots per key tile
constexpr uint32_t kHalfBytes = BN * 128;    // 128 rows x 64 bf16, 128-byte swizzle
constexpr uint32_t kTileBytes = 2 * kHalfBytes;
constexpr int kRowBlock = 256;               // rows per walk: columns of an S^T buffer
constexpr uint32_t kQHalfBytes = kRowBlock * 128;
constexpr int kStages = 4;
enum {
  W_FULL = 0,
  W_EMPTY = W_FULL + kStages,
  W_QREADY = W_EMPTY + kStages,
  W_SFULL,                     // [buffer][half of the columns]
  W_SEMPTY = W_SFULL + 4,
  W_XSUM = W_SEMPTY + 4,       // [buffer][tile parity][lane quarter]: the upper columns' sums written
  W_DONE = W_XSUM + 16,        // the sixteen warps have finished a walk
  W_FINAL,
  W_TEARDOWN,
  W_COUNT
};
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_RING = 2 * kQHalfBytes;
constexpr uint32_t OFF_ONES = OFF_RING + kStages * kTileBytes;     // the statistics' operands, 16 columns, not swizzled:
constexpr uint32_t OFF_BIAS = OFF_ONES + BN * 32;                  //   ones for each slot; -M and -log l for each row
constexpr uint32_t OFF_SEE = OFF_BIAS + 2 * kRowBlock * 32;        // per drafted token: those it sees
constexpr uint32_t OFF_XSUM = OFF_SEE + kMaxDrafts * 8;            // [buffer][tile parity][slot]
constexpr uint32_t OFF_BAR = OFF_XSUM + 4 * BN * 4;
constexpr uint32_t OFF_LINE = OFF_BAR + 8 * ((W_COUNT + 1) & ~1);
constexpr uint32_t OFF_TMEMPTR = OFF_LINE + sizeof(Line);
constexpr uint32_t OFF_ABORT = OFF_TMEMPTR + 4;
constexpr uint32_t kSmemAlloc = OFF_ABORT + 8 + 1024;
static_assert(kSmemAlloc <= 227 * 1024, "shared memory budget");
static_assert(BN == kTileSlots, "the line is cut into these tiles");

// byte offset of element (row, k) of a 16-column bf16 operand without swizzle
__device__ __forceinline__ uint32_t noswz_off(int row, int k) {
  return (uint32_t)((row >> 3) * 256 + (k >> 3) * 128 + (row & 7) * 16 + (k & 7) * 2);
}
// an fp32 value as the sum of three bf16 values, 8 significant bits each
__device__ __forceinline__ void write_parts(unsigned char* at, float x) {
  const __nv_bfloat16 hi = __float2bfloat16(x);
  const float r1 = x - __bfloat162float(hi);
  const __nv_bfloat16 mid = __float2bfloat16(r1);
  const __nv_bfloat16 lo = __float2bfloat16(r1 - __bfloat162float(mid));
  __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(at);
  d[0] = hi;
  d[1] = mid;
  d[2] = lo;
}

__global__ void __launch_bounds__(kThreads, 1) tree_weight_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                  const TreeParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
  Line* line = reinterpret_cast<Line*>(smem + OFF_LINE);
  uint64_t* see = reinterpret_cast<uint64_t*>(smem + OFF_SEE);
  float* xsum = reinterpret_cast<float*>(smem + OFF_XSUM);
  auto bar = [&](int i) { return sbase + OFF_BAR + 8u * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (warp == 0) {
    if (lane == 0) {
      abort_flag[0] = 0;
      abort_flag[1] = p.hold ? 1 << p.hold : (int)kWaitLimitNs;
      for (int s = 0; s < kStages; ++s) {
        mbar_init(bar(W_FULL + s), 1);
        mbar_init(bar(W_EMPTY + s), 1);
      }
      mbar_init(bar(W_QREADY), 16);
      for (int s = 0; s < 4; ++s) {
        mbar_init(bar(W_SFULL + s), 1);
        mbar_init(bar(W_SEMPTY + s), 4);
      }
      for (int s = 0; s < 16; ++s) mbar_init(bar(W_XSUM + s), 1);
      mbar_init(bar(W_DONE), 16);
      mbar_init(bar(W_FINAL), 1);
      mbar_init(bar(W_TEARDOWN), kThreads / 32 - 1);
      fence_mbar_init();
      prefetch_tmap(&kmap);
    }
  } else if (warp == 1) {
    tmem_alloc(sbase + OFF_TMEMPTR, kTmemCols);
    tmem_relinquish();
  } else if (warp == 2) {
    const Line L = find_share(p, blockIdx.x, lane);
    if (lane == 0) *line = L;
  }
  for (uint32_t o = threadIdx.x * 16; o < OFF_SEE - OFF_ONES; o += kThreads * 16)
    *reinterpret_cast<uint4*>(smem + OFF_ONES + o) = make_uint4(0, 0, 0, 0);
  __syncthreads();
  for (int i = threadIdx.x; i < 3 * BN; i += kThreads)
    *reinterpret_cast<__nv_bfloat16*>(smem + OFF_ONES + noswz_off(i / 3, i % 3)) = __float2bfloat16(1.f);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEMPTR), 0);
  const Waits wait{abort_flag, p.status};
  Pieces walk{line->start, line->end, line->base, line->b};
  Piece w{};
  const int walks = (p.rows + kRowBlock - 1) / kRowBlock;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t g = 0;
      bool ok = p.hold == 0;
      const uint64_t usual = l2_evict_normal(), last = l2_evict_first();
      while (ok && walk.next(p, &w)) {
        for (int rb = 0; ok && rb < walks; ++rb)
          for (int i = 0; i < w.n; ++i, ++g) {
            const uint32_t st = g % kStages;
            if (g >= kStages && !wait(bar(W_EMPTY + st), (g / kStages - 1) & 1)) {
              ok = false;
              break;
            }
            const uint32_t dst = sbase + OFF_RING + st * kTileBytes;
            mbar_arrive_expect_tx(bar(W_FULL + st), kTileBytes);
            // the last walk over a tile needs it no longer
            const uint64_t policy = rb == walks - 1 ? last : usual;
            tma_load_4d(dst, &kmap, bar(W_FULL + st), 0, (w.t0 + i) * BN, w.h, w.b, policy);
            tma_load_4d(dst + kHalfBytes, &kmap, bar(W_FULL + st), 64, (w.t0 + i) * BN, w.h, w.b, policy);
          }
      }
      for (uint32_t q = g > kStages ? g - kStages : 0; q < g; ++q)
        mbar_wait(bar(W_FULL + q % kStages), (q / kStages) & 1, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // the whole warp runs the loop and an elected lane issues, as in tree_attn.cu
    auto wait_all = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)); };
    uint32_t g = 0, used[2] = {0, 0}, n_q = 0;
    bool ok = true;
    while (ok && walk.next(p, &w)) {
      const int n = __shfl_sync(0xffffffffu, w.n, 0);
      for (int rb = 0; ok && rb < walks; ++rb) {
        if (!(ok = wait_all(bar(W_QREADY), n_q++ & 1))) break;
        const int n_rows = min(p.rows - rb * kRowBlock, kRowBlock);
        // each half of the columns on its own: its warps free it on their own
        const int n_half = ((n_rows + 31) & ~31) / 2;
        const uint32_t idesc = idesc_bf16_f32(BN, n_half, false);
        for (int i = 0; ok && i < n; ++i, ++g) {
          const int s = i & 1;
          const uint32_t st = g % kStages;
          if (!(ok = wait_all(bar(W_FULL + st), (g / kStages) & 1))) break;
          const uint64_t ka = smem_desc_sw128(sbase + OFF_RING + st * kTileBytes, 16, 1024);
          for (int half = 0; half < 2; ++half) {
            if (used[s] > 0 && !(ok = wait_all(bar(W_SEMPTY + 2 * s + half), (used[s] - 1) & 1))) break;
            tc_fence_after();
            const uint32_t d = tmem + s * 256 + half * n_half;
            const uint64_t qa = smem_desc_sw128(sbase + OFF_Q + half * n_half * 128, 16, 1024);
            const uint64_t ones = smem_desc_noswz(sbase + OFF_ONES, 128, 256);
            const uint64_t bias = smem_desc_noswz(sbase + OFF_BIAS + half * n_half * 32, 128, 256);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_ss(d, ka + (((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4),
                       qa + (((k >> 2) * kQHalfBytes + (k & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
              // S - M first, as an exact difference of like numbers, then - log l
#pragma unroll
              for (int k = 0; k < 2; ++k) mma_ss(d, ones, bias + (k * kRowBlock * 32 >> 4), idesc, 1u);
              mma_commit(bar(W_SFULL + 2 * s + half));
              if (half == 1) mma_commit(bar(W_EMPTY + st));
            }
            __syncwarp();
          }
          if (!ok) break;
          ++used[s];
        }
      }
    }
    if (elect_one()) mma_commit(bar(W_FINAL));
    mbar_wait(bar(W_FINAL), 0, kWaitLimitNs);
  } else if (warp >= 4) {
    // per S^T buffer two groups of four warps, one for each half of the columns
    const int buf = ((warp - 4) >> 2) & 1, upper = (warp - 4) >> 3, quarter = warp & 3, key = quarter * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 256;
    const float c = p.scale_log2;
    const uint64_t c2 = pk2(c, c);
    uint32_t n_s = 0, n_done = 0;
    bool ok = true;
    wait_for_predecessors();       // the rows' statistics come from the attention
    while (ok && walk.next(p, &w)) {
      const long long row_base = ((long long)w.b * p.Hq + (long long)w.h * p.G) * p.T;
      const int slots = w.len + w.draft;
      const bool tail = (w.t0 + w.n) * BN > w.len;
      const float* w_in = p.weight + ((long long)w.b * p.Hkv + w.h) * p.cap;
      float* w_out = p.weight_out + ((long long)w.b * p.Hkv + w.h) * p.cap;
      if (tail) {      // the same values from every warp
        const Sees sv = tree_sees(p, w.b, w.draft, lane);
        see[lane] = sv.m0;
        see[lane + 32] = sv.m1;
      }
      for (int rb = 0; ok && rb < walks; ++rb) {
        // the Q operand and the row statistics: 16 rows per warp. Rows past
        // the end and of missing tokens are zeros with weight 0.
        const int n_rows = min(p.rows - rb * kRowBlock, kRowBlock), n_pad = (n_rows + 31) & ~31;
        const int ch = lane & 15;
        uint4 v[8];
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int at = (warp - 4) * 16 + it * 2 + (lane >> 4), r = rb * kRowBlock + at;
          v[it] = make_uint4(0, 0, 0, 0);
          if (at < n_rows && r % p.T < w.draft)
            v[it] = *reinterpret_cast<const uint4*>(p.Q + (row_base + r) * kHeadDim + ch * 8);
        }
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int at = (warp - 4) * 16 + it * 2 + (lane >> 4);
          if (at < n_pad)
            *reinterpret_cast<uint4*>(smem + OFF_Q + (ch >> 3) * kQHalfBytes + at * 128 +
                                      (((ch & 7) ^ (at & 7)) << 4)) = v[it];
        }
        if (lane < 16) {
          const int at = (warp - 4) * 16 + lane, r = rb * kRowBlock + at;
          float minus_m = -INFINITY, minus_log = 0.f;
          if (at < n_rows && r % p.T < w.draft) {
            const float2 st = p.row_stat[row_base + r];
            minus_m = -st.x;
            minus_log = __log2f(st.y) / c;
          }
          if (at < n_pad) {
            unsigned char* m_at = smem + OFF_BIAS + noswz_off(at, 0);
            if (minus_m == -INFINITY) {      // no inf - inf in the lower parts
              *reinterpret_cast<uint2*>(m_at) = make_uint2(0xFF80u, 0u);
            } else {
              write_parts(m_at, minus_m);
            }
            write_parts(m_at + kRowBlock * 32, minus_log);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(W_QREADY));

        for (int i = buf; i < w.n; i += 2) {
          const int slot = (w.t0 + i) * BN + key;
          const bool live = slot < slots;
          float old = 0.f;
          if (live && !upper) old = rb > 0 ? w_out[slot] : slot < w.len ? w_in[slot] : 0.f;
          if (!(ok = wait(bar(W_SFULL + 2 * buf + upper), n_s & 1))) break;
          ++n_s;
          tc_fence_after();
          const int d = slot - w.len;                // drafted token of the slot
          // which tokens see this slot, and the token of the walk's first row
          uint64_t seen = ~0ull;
          const bool masked = (w.t0 + i + 1) * BN > w.len;
          if (masked && d >= 0) {
            seen = 0;
            for (int t = 0; t < w.draft; ++t) seen |= ((see[t] >> (d & 63)) & 1) << t;
          }
          const int n_half = n_pad / 2, col0 = upper * n_half;      // this warp's columns
          int t = (rb * kRowBlock + col0) % p.T;
          uint64_t acc[2] = {0ull, 0ull};
          // 16 rows: their p, added in pairs
          auto add = [&](auto with_mask, const uint32_t (&s)[16]) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float x0, x1;
              unpk2(mul2(pk2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2), x0, x1);
              x0 = fast_exp2(x0);
              x1 = fast_exp2(x1);
              if (with_mask.value) {
                x0 = (seen >> t) & 1 ? x0 : 0.f;
                t = t + 1 == p.T ? 0 : t + 1;
                x1 = (seen >> t) & 1 ? x1 : 0.f;
                t = t + 1 == p.T ? 0 : t + 1;
              }
              acc[(e >> 1) & 1] = add2(acc[(e >> 1) & 1], pk2(x0, x1));
            }
          };
          // the next 16 columns are on their way while these are added
          auto add_all = [&](auto with_mask) {
            uint32_t s0[16], s1[16];
            tmem_ld16(tS + col0, s0);
            tmem_wait_ld();
#pragma unroll 1
            for (int r0 = 0; r0 < n_half; r0 += 32) {
              if (r0 + 16 < n_half) tmem_ld16(tS + col0 + r0 + 16, s1);
              add(with_mask, s0);
              if (r0 + 16 >= n_half) break;
              tmem_wait_ld();
              if (r0 + 32 < n_half) tmem_ld16(tS + col0 + r0 + 32, s0);
              add(with_mask, s1);
              tmem_wait_ld();
            }
          };
          if (masked) add_all(std::true_type{});
          else add_all(std::false_type{});
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(W_SEMPTY + 2 * buf + upper));
          float a0, a1;
          unpk2(add2(acc[0], acc[1]), a0, a1);
          // the lower columns' warp adds the upper columns' sums and writes
          const int x = buf * 2 + (int)((n_s - 1) & 1);
          if (upper) {
            xsum[x * BN + key] = a0 + a1;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(W_XSUM + x * 4 + quarter));
          } else {
            if (!(ok = wait(bar(W_XSUM + x * 4 + quarter), ((n_s - 1) >> 1) & 1))) break;
            if (live) w_out[slot] = old + (a0 + a1 + xsum[x * BN + key]);
          }
        }
        if (!ok) break;
        // Q and the statistics may change once every warp is done with them
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(W_DONE));
        if (!(ok = wait(bar(W_DONE), n_done & 1))) break;
        ++n_done;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  if (warp != 1) {
    if (lane == 0) mbar_arrive(bar(W_TEARDOWN));
    return;
  }
  mbar_wait(bar(W_TEARDOWN), 0, kWaitLimitNs);
  __syncwarp();
  tc_fence_after();
  tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

int launch_tree_weight(const CUtensorMap& k, const TreeParams& p, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  int dev = 0, sms = 0;
  cudaError_t e = this_device(&dev, &sms);
  if (e == cudaSuccess) e = allow_smem(tree_weight_kernel, (int)kSmemAlloc, dev, done);
  if (e != cudaSuccess) return cuda_status(e);
  return launch_after(tree_weight_kernel, dim3(p.grid), dim3(kThreads), kSmemAlloc, stream, k, p);
}

}  // namespace dhsa
