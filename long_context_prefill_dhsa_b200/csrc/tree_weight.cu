// Attention weight of each cache slot: weight_out = weight + sum over the rows
// (query heads of the group x drafted tokens) of p = exp(scale (s - M)) / l,
// with each row's largest score M and denominator l from the attention.
//
// The scores are computed again, transposed: S^T = K Q^T puts the slots on the
// tensor core's M side, so that a thread owns a TMEM lane, one slot, and adds
// its rows' p with no exchange between threads. K is read once more (256
// bytes per slot); up to about 180 rows that read is the bound, above them
// the exponentials (16 per cycle and SM).
//
// Warp 0 streams the K tiles, warp 1 issues the MMAs into two S^T buffers of
// 256 columns, warps 4 to 7 take the even and warps 8 to 11 the odd tiles.
// More than 256 rows walk the same keys again and add to weight_out.
// Waits are bounded as in tree_attn.cu.
#include "tree.cuh"

namespace dhsa {
namespace {

constexpr int kThreads = 384;
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
  W_SFULL,                     // per buffer
  W_SEMPTY = W_SFULL + 2,
  W_DONE = W_SEMPTY + 2,       // the eight warps have finished a walk
  W_FINAL,
  W_TEARDOWN,
  W_COUNT
};
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_RING = 2 * kQHalfBytes;
constexpr uint32_t OFF_STAT = OFF_RING + kStages * kTileBytes;     // float4 per pair of rows: -M0, -M1, 1/l0, 1/l1
constexpr uint32_t OFF_SEE = OFF_STAT + kRowBlock / 2 * 16;        // per row: drafted tokens it sees
constexpr uint32_t OFF_BAR = OFF_SEE + kRowBlock * 8;
constexpr uint32_t OFF_LINE = OFF_BAR + 8 * ((W_COUNT + 1) & ~1);
constexpr uint32_t OFF_TMEMPTR = OFF_LINE + sizeof(Line);
constexpr uint32_t OFF_ABORT = OFF_TMEMPTR + 4;
constexpr uint32_t kSmemAlloc = OFF_ABORT + 4 + 1024;
static_assert(kSmemAlloc <= 227 * 1024, "shared memory budget");

__global__ void __launch_bounds__(kThreads, 1) tree_weight_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                  const TreeParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
  Line* line = reinterpret_cast<Line*>(smem + OFF_LINE);
  float4* stat = reinterpret_cast<float4*>(smem + OFF_STAT);
  uint64_t* see = reinterpret_cast<uint64_t*>(smem + OFF_SEE);
  auto bar = [&](int i) { return sbase + OFF_BAR + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {
    if (lane == 0) {
      *abort_flag = 0;
      for (int s = 0; s < kStages; ++s) {
        mbar_init(bar(W_FULL + s), 1);
        mbar_init(bar(W_EMPTY + s), 1);
      }
      mbar_init(bar(W_QREADY), 8);
      for (int s = 0; s < 2; ++s) {
        mbar_init(bar(W_SFULL + s), 1);
        mbar_init(bar(W_SEMPTY + s), 4);
      }
      mbar_init(bar(W_DONE), 8);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEMPTR);
  const Waits wait{abort_flag, p.status};
  Pieces walk{line->start, line->end, line->base, line->b};
  Piece w{};
  const int walks = (p.rows + kRowBlock - 1) / kRowBlock;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t g = 0;
      bool ok = true;
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
            tma_load_4d(dst, &kmap, bar(W_FULL + st), 0, (w.t0 + i) * BN, w.h, w.b);
            tma_load_4d(dst + kHalfBytes, &kmap, bar(W_FULL + st), 64, (w.t0 + i) * BN, w.h, w.b);
          }
      }
      for (uint32_t q = g > kStages ? g - kStages : 0; q < g; ++q)
        mbar_wait(bar(W_FULL + q % kStages), (q / kStages) & 1, kWaitLimitNs);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t g = 0, used[2] = {0, 0}, n_q = 0;
      bool ok = true;
      while (ok && walk.next(p, &w)) {
        for (int rb = 0; ok && rb < walks; ++rb) {
          if (!(ok = wait(bar(W_QREADY), n_q++ & 1))) break;
          const int n_rows = min(p.rows - rb * kRowBlock, kRowBlock);
          const uint32_t idesc = idesc_bf16_f32(BN, (n_rows + 15) & ~15, false);
          for (int i = 0; i < w.n; ++i, ++g) {
            const int s = i & 1;
            const uint32_t st = g % kStages;
            if (!(ok = wait(bar(W_FULL + st), (g / kStages) & 1))) break;
            if (used[s] > 0 && !(ok = wait(bar(W_SEMPTY + s), (used[s] - 1) & 1))) break;
            ++used[s];
            tc_fence_after();
            const uint32_t ka = sbase + OFF_RING + st * kTileBytes;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t c = (k & 3) * 32;
              mma_ss(tmem + s * 256, smem_desc_sw128(ka + (k >> 2) * kHalfBytes + c, 16, 1024),
                     smem_desc_sw128(sbase + OFF_Q + (k >> 2) * kQHalfBytes + c, 16, 1024), idesc, k > 0 ? 1u : 0u);
            }
            mma_commit(bar(W_SFULL + s));
            mma_commit(bar(W_EMPTY + st));
          }
        }
      }
      mma_commit(bar(W_FINAL));
      mbar_wait(bar(W_FINAL), 0, kWaitLimitNs);
    }
  } else if (warp >= 4) {
    const int buf = (warp - 4) >> 2, quarter = warp & 3, key = quarter * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 256;
    const float c = p.scale_log2;
    const uint64_t c2 = pk2(c, c);
    uint32_t n_s = 0, n_done = 0;
    bool ok = true;
    while (ok && walk.next(p, &w)) {
      const long long row_base = ((long long)w.b * p.Hq + (long long)w.h * p.G) * p.T;
      const int slots = w.len + w.draft;
      const bool tail = (w.t0 + w.n) * BN > w.len;
      const float* w_in = p.weight + ((long long)w.b * p.Hkv + w.h) * p.cap;
      float* w_out = p.weight_out + ((long long)w.b * p.Hkv + w.h) * p.cap;
      Sees sv{0, 0};
      if (tail) sv = tree_sees(p, w.b, w.draft, lane);
      for (int rb = 0; ok && rb < walks; ++rb) {
        // the Q operand and the row statistics: 32 rows per warp. Rows past
        // the end and of missing tokens are zeros with weight 0.
        const int n_rows = min(p.rows - rb * kRowBlock, kRowBlock), n_pad = (n_rows + 15) & ~15;
        const int ch = lane & 15;
#pragma unroll
        for (int half = 0; half < 2; ++half) {       // eight loads in flight
          uint4 v[8];
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const int at = (warp - 4) * 32 + half * 16 + it * 2 + (lane >> 4), r = rb * kRowBlock + at;
            v[it] = make_uint4(0, 0, 0, 0);
            if (at < n_rows && r % p.T < w.draft)
              v[it] = *reinterpret_cast<const uint4*>(p.Q + (row_base + r) * kHeadDim + ch * 8);
          }
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const int at = (warp - 4) * 32 + half * 16 + it * 2 + (lane >> 4);
            if (at < n_pad)
              *reinterpret_cast<uint4*>(smem + OFF_Q + (ch >> 3) * kQHalfBytes + at * 128 +
                                        (((ch & 7) ^ (at & 7)) << 4)) = v[it];
          }
        }
        {
          const int at = (warp - 4) * 32 + lane, r = rb * kRowBlock + at;
          const int t = r % p.T;
          const uint64_t sees = sv.of(t);
          float2 st = make_float2(0.f, 0.f);
          if (at < n_rows && t < w.draft) st = p.row_stat[row_base + r];
          float* f = reinterpret_cast<float*>(stat + at / 2);
          f[at & 1] = -st.x;
          f[2 + (at & 1)] = st.y;
          see[at] = sees;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(W_QREADY));
        // the statistics are read by all eight warps
        if (!(ok = wait(bar(W_QREADY), n_done & 1))) break;

        for (int i = buf; i < w.n; i += 2) {
          const int slot = (w.t0 + i) * BN + key;
          const bool live = slot < slots;
          float old = 0.f;
          if (live) old = rb > 0 ? w_out[slot] : slot < w.len ? w_in[slot] : 0.f;
          if (!(ok = wait(bar(W_SFULL + buf), n_s & 1))) break;
          ++n_s;
          tc_fence_after();
          const bool masked = (w.t0 + i + 1) * BN > w.len;
          const int d = slot - w.len;                // drafted token of the slot
          uint64_t acc = 0ull;
          float acc1 = 0.f;
          for (int r0 = 0; r0 < n_pad; r0 += 16) {
            uint32_t s[16];
            tmem_ld16(tS + r0, s);
            tmem_wait_ld();
            if (!masked) {
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float4 st = stat[(r0 + e) / 2];
                const uint64_t x = mul2(add2(pk2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), pk2(st.x, st.y)), c2);
                float x0, x1;
                unpk2(x, x0, x1);
                acc = fma2(pk2(fast_exp2(x0), fast_exp2(x1)), pk2(st.z, st.w), acc);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float* f = reinterpret_cast<const float*>(stat + (r0 + e) / 2);
                if (d < 0 || ((see[r0 + e] >> (d & 63)) & 1))
                  acc1 += fast_exp2((__uint_as_float(s[e]) + f[e & 1]) * c) * f[2 + (e & 1)];
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(W_SEMPTY + buf));
          float a0, a1;
          unpk2(acc, a0, a1);
          if (live) w_out[slot] = old + (a0 + a1 + acc1);
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

int tree_weight_tile() { return BN; }

int launch_tree_weight(const CUtensorMap& k, const TreeParams& p, cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(tree_weight_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemAlloc);
  if (e != cudaSuccess) return cuda_status(e);
  tree_weight_kernel<<<p.grid, kThreads, kSmemAlloc, stream>>>(k, p);
  return launch_status();
}

}  // namespace dhsa
