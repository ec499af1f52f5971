// Attention of drafted tokens over a key/value cache.
//
// Token t of sequence b sees the cached slots s < len, itself and its
// ancestors in the drafted tree; O = softmax(scale q k) v over them.
//
// The G query heads of a kv head and their T tokens read the same keys, so
// their G*T rows (contiguous in Q) are one matrix operand, and each key and
// value is read from HBM once: 512 bytes per slot against 512 FLOP per slot
// and row. Up to about 250 rows HBM is the bound, above them the tensor cores
// and the exponentials. Measured (32/8 heads, joining included): one token over
// 131071 slots 89.6 us, 537 MB at 6.0 TB/s; 64 tokens over 131008 slots 145 us,
// 137 GFLOP at 945 TFLOP/s, where each stream waits in turn for its scores and
// for its exponentials (over 40000 slots tensor cores 41% busy, special-function units 42%).
//
// sm_100a design
// --------------
// * Work: the 128-slot key tiles of all (sequence, kv head, query block) items
//   are one line, cut into shares, one per CTA of a persistent grid (tree.cuh):
//   parts of one item each while there are CTAs for every item, equal shares
//   of the line beyond that. Lengths are read on the device, so ragged batches balance
//   without host help. A CTA that has all of an item writes its rows; the
//   others leave an unnormalised O with its reference score and sum for each
//   piece, and a second kernel joins an item's pieces.
// * Two softmax streams per CTA, each with its own S and O in TMEM (4 x 128
//   columns) and its own warps. With up to 128 rows they take the even
//   and the odd key tiles of the same query tile; with more they take two
//   query tiles over the same key tiles. While one stream does its
//   exponentials the tensor core works for the other, and each half of P
//   goes to the tensor core while the softmax does the other half.
// * Warp 0 streams K and V tiles (TMA, 32 KB each) into one ring; warp 1
//   issues S = Q K^T (both operands in shared memory) and O += P V (P from
//   TMEM, over the S it came from); the warps from 4 on are the streams' softmax.
//   A single issuer keeps the tensor operations in order.
// * Query row r sits in TMEM lane 32 (r mod 4) + r / 4, so that few rows (one
//   token: G of them) spread over all four lane quarters, and the shape
//   16x256b gives each row to four threads.
// * P is rounded to bf16 for the tensor core, as V is bf16 and both operands
//   share a type; the row sum adds the fp32 values.
// * Slots past the last one can hold anything: their scores are replaced, and
//   their V rows are zeroed in shared memory (0 x NaN would be NaN).
// * Every wait is bounded; a timeout raises DHSA_DEVFLAG_WAIT_TIMEOUT, and the
//   CTA drains its copies and MMAs, frees its TMEM and exits.
#include "tree.cuh"

namespace dhsa {

int launch_tree_join(const TreeParams& p, cudaStream_t stream);
int launch_tree_join_weights(const TreeParams& p, cudaStream_t stream);
int launch_tree_weight(const CUtensorMap& k, const TreeParams& p, cudaStream_t stream);

namespace {

// producer, issuer, two helpers, and the softmax: eight warps for each half of the lanes of a quarter in use
constexpr int block_threads(int halves) { return 128 + 256 * halves; }
constexpr int BM = 128;          // query rows per tile
constexpr int BN = 128;          // slots per key tile
constexpr uint32_t kHalfBytes = BM * 128;    // 128 query rows x 64 bf16, 128-byte swizzle
constexpr uint32_t kTileBytes = 2 * kHalfBytes;
constexpr uint32_t kKvHalfBytes = BN * 128;
constexpr uint32_t kKvBytes = 2 * kKvHalfBytes;
// Items of short caches are not split: a CTA takes whole ones and writes O
// itself, which saves the joining kernel and, with many items, the draining
// and refilling of the pipeline. Whole against split, us, 32/8 heads, one token:
//   500 slots:  1 sequence 10.3 / 10.9, 8 sequences 10.9 / 12.3, 64 sequences 34 / 38
//   600 slots:  1 sequence 11.0 / 10.9, 8 sequences 11.8 / 13.1, 32 sequences 23 / 26
//   1000 slots: 1 sequence 14.2 / 10.3, 4 sequences 14.4 / 13.0, 8 sequences 15.0 / 15.8, 32 sequences 30 / 32
//   2000 slots: 1 sequence 22 / 11, 8 sequences 23 / 21, 64 sequences 94 / 90
constexpr int kWholeTiles = 5;        // with any number of items
constexpr int kWholeTilesMany = 8;    // with at least kManyItems, two fifths of the CTAs
constexpr int kManyItems = 64;
constexpr float kRaise = 20.f, kTop = 1048576.f;   // powers of two by which a score may pass its row's reference; its p
constexpr uint32_t kSmemData = 224 * 1024;   // query tiles (one or two of 32 KB), the rest is the ring of K and V tiles
constexpr int kMaxStages = (kSmemData - kTileBytes) / kKvBytes;

struct TreeMaps {
  CUtensorMap k, v;
};

// shared memory after the tiles
enum {
  B_FULL = 0,                   // ring stage holds its tile
  B_EMPTY = B_FULL + kMaxStages,
  B_QREADY = B_EMPTY + kMaxStages,
  B_SFULL,                      // per stream: S complete
  B_PREADY = B_SFULL + 2,       // [stream][half]: P of 64 slots written
  B_PVHALF = B_PREADY + 4,      // per stream: P V of a tile's first half complete
  B_OFINAL = B_PVHALF + 2,      // every MMA of the piece complete
  B_XCHG,                       // per lane quarter and half: stream 1's references and sums written
  B_FINAL = B_XCHG + 8,
  B_TEARDOWN,
  B_COUNT
};
constexpr uint32_t OFF_BAR = kSmemData;
constexpr uint32_t OFF_SEE = OFF_BAR + 8 * ((B_COUNT + 1) & ~1);   // drafted tokens that each drafted token sees
constexpr uint32_t OFF_XCHG = OFF_SEE + kMaxDrafts * 8;            // per row of the tile: stream 1's reference and sum
constexpr uint32_t OFF_LINE = OFF_XCHG + BM * 8;
constexpr uint32_t OFF_TMEMPTR = OFF_LINE + sizeof(Line);
constexpr uint32_t OFF_ABORT = OFF_TMEMPTR + 4;
constexpr uint32_t kSmemAlloc = OFF_ABORT + 8 + 1024;   // slack for aligning the base
static_assert(kSmemAlloc <= 227 * 1024, "shared memory budget");
static_assert(sizeof(Line) % 8 == 0, "alignment");
static_assert(BN == kTileSlots && BM == kTileRows, "the line is cut into these tiles");

constexpr int W_PRODUCER = 0, W_MMA = 1, W_SOFTMAX0 = 4;

// NQT: query tiles per CTA. HALVES: lane halves in use (one: up to 64 rows).
template <int NQT, int HALVES>
__global__ void __launch_bounds__(block_threads(HALVES), 1) tree_attn_kernel(const __grid_constant__ TreeMaps maps,
                                                                const TreeParams p) {
  constexpr int kThreads = block_threads(HALVES), kStreamWarps = 4 * HALVES;
  // rows of the MMAs: with 64, their D lies in the first 16 lanes of each quarter
  constexpr int MQ = 64 * HALVES, kQBits = 5 + HALVES, kLanes = 16 * HALVES;
  constexpr uint32_t kQHalf = MQ * 128, kQTile = 2 * kQHalf;
  constexpr int NST = (kSmemData - NQT * kQTile) / kKvBytes;   // ring stages
  constexpr int kAhead = 2 / NQT;   // tiles whose scores are computed ahead: one S for each of two streams
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ring = sbase + NQT * kQTile;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
  Line* line = reinterpret_cast<Line*>(smem + OFF_LINE);
  auto bar = [&](int i) { return sbase + OFF_BAR + 8u * i; };
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (warp == W_PRODUCER && lane == 0) {
    abort_flag[0] = 0;
    abort_flag[1] = p.hold ? 1 << p.hold : (int)kWaitLimitNs;
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    mbar_init(bar(B_QREADY), 2 * kStreamWarps);
    for (int s = 0; s < 4; ++s) mbar_init(bar(B_PREADY + s), kStreamWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_SFULL + s), 1);
      mbar_init(bar(B_PVHALF + s), 1);
    }
    mbar_init(bar(B_OFINAL), 1);
    for (int s = 0; s < 8; ++s) mbar_init(bar(B_XCHG + s), 1);
    mbar_init(bar(B_FINAL), 1);
    mbar_init(bar(B_TEARDOWN), kThreads / 32 - 1);
    fence_mbar_init();
  }
  __syncthreads();
  // The producer needs nothing but the barriers and its share: it starts the
  // copies while the others allocate TMEM and look up theirs.
  Line share;
  uint32_t tmem = 0;
  if (warp == W_PRODUCER) {
    share = find_share(p, blockIdx.x, lane);
  } else {
    if (warp == W_MMA) {
      tmem_alloc(sbase + OFF_TMEMPTR, kTmemCols);
      tmem_relinquish();
    } else if (warp == 2) {
      share = find_share(p, blockIdx.x, lane);
      if (lane == 0) *line = share;
    } else if (warp == 3 && blockIdx.x == 0) {
      bool bad = false;
      for (int b = lane; b < p.B; b += 32) bad |= seq_len(p.lengths, p.n_draft, p.T, b, p.T, p.cap).bad;
      if (bad) raise_device_flag(p.status, DHSA_DEVFLAG_BAD_CACHE);
    }
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 32) : "memory");
    tc_fence_after();
    tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEMPTR), 0);
    share = *line;
  }
  const Waits wait{abort_flag, p.status};
  Pieces walk{share.start, share.end, share.base, share.b};
  Piece w{};

  if (warp == W_PRODUCER) {
    if (lane == 0) {
      // keys and values are read once (per query block) and must not push
      // everything else out of L2; K stays where the weight pass reads it again
      const uint64_t v_policy = p.blocks > 1 ? l2_evict_normal() : l2_evict_first();
      const uint64_t k_policy = p.keep_k || p.blocks > 1 ? l2_evict_normal() : l2_evict_first();
      uint32_t g = 0;     // tiles loaded
      bool ok = p.hold == 0;
      auto load = [&](const CUtensorMap* m, int tile) {
        const uint32_t st = g % NST;
        if (g >= NST && !wait(bar(B_EMPTY + st), (g / NST - 1) & 1)) return false;
        const uint32_t dst = ring + st * kKvBytes;
        mbar_arrive_expect_tx(bar(B_FULL + st), kKvBytes);
        const uint64_t policy = m == &maps.k ? k_policy : v_policy;
        tma_load_4d(dst, m, bar(B_FULL + st), 0, tile * BN, w.h, w.b, policy);
        tma_load_4d(dst + kKvHalfBytes, m, bar(B_FULL + st), 64, tile * BN, w.h, w.b, policy);
        ++g;
        return true;
      };
      while (ok && walk.next(p, &w)) {
        // the order in which the issuer uses them: K tiles kAhead before V tiles
        for (int i = 0; ok && i < kAhead && i < w.n; ++i) ok = load(&maps.k, w.t0 + i);
        for (int i = 0; ok && i < w.n; ++i) {
          ok = load(&maps.v, w.t0 + i);
          if (ok && i + kAhead < w.n) ok = load(&maps.k, w.t0 + i + kAhead);
        }
      }
      // copies in flight must land before the CTA ends
      for (uint32_t q = g > NST ? g - NST : 0; q < g; ++q) mbar_wait(bar(B_FULL + q % NST), (q / NST) & 1, kWaitLimitNs);
    }
  } else if (warp == W_MMA) {
    // The whole warp runs the loop, and an elected lane issues: operands then
    // live in uniform registers. (With the loop in one lane, or the lane as
    // each instruction's predicate, an MMA took 105 to 120 cycles to issue
    // beside the busy softmax warps, against 65 to execute.)
    const uint32_t idesc_qk = idesc_bf16_f32(MQ, BN, false), idesc_pv = idesc_bf16_f32(MQ, kHeadDim, true);
    const uint64_t q_desc = smem_desc_sw128(sbase, 16, 1024), k_desc = smem_desc_sw128(ring, 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(ring, kKvHalfBytes, 1024);
    uint32_t g = 0, n_piece = 0, p_phase = 0;    // p_phase: parity of P's barriers, a bit for each stream
    auto wait_all = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)); };
    auto empty = [&](uint32_t q) { return bar(B_EMPTY + q % NST); };
    auto commit = [&](uint32_t b) {
      if (elect_one()) mma_commit(b);
      __syncwarp();
    };
    auto qk = [&](int s, uint32_t q, bool done) {      // S = Q K^T; done: the K tile's last use
      const uint64_t qa = q_desc + (NQT == 2 ? s * (kQTile >> 4) : 0), ka = k_desc + q % NST * (kKvBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ss(tmem + s * 128, qa + (((k >> 2) * kQHalf + (k & 3) * 32) >> 4),
                 ka + (((k >> 2) * kKvHalfBytes + (k & 3) * 32) >> 4), idesc_qk, k > 0 ? 1u : 0u);
        mma_commit(bar(B_SFULL + s));
        if (done) mma_commit(empty(q));
      }
      __syncwarp();
    };
    auto arrived = [&](uint32_t q) {
      const bool ok = wait_all(bar(B_FULL + q % NST), (q / NST) & 1);
      tc_fence_after();
      return ok;
    };
    // O += P V, each half as soon as its P is there; done: the V tile's last use
    auto pv = [&](int s, uint32_t q, bool first, bool done) {
      const uint64_t va = v_desc + q % NST * (kKvBytes >> 4);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!wait_all(bar(B_PREADY + 2 * s + half), (p_phase >> s) & 1)) return false;
        if (half == 0 && !wait_all(bar(B_FULL + q % NST), (q / NST) & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 4 * half; k < 4 * half + 4; ++k)
            mma_ts(tmem + 256 + s * 128, tmem + s * 128 + k * 8, va + k * (2048 >> 4), idesc_pv,
                   (!first || k > 0) ? 1u : 0u);
          if (half == 0) mma_commit(bar(B_PVHALF + s));
          else if (done) mma_commit(empty(q));
        }
        __syncwarp();
      }
      p_phase ^= 1u << s;
      return true;
    };
    bool ok = true;
    while (ok && walk.next(p, &w)) {
      const int n = __shfl_sync(0xffffffffu, w.n, 0);
      if (!wait_all(bar(B_QREADY), n_piece & 1)) break;
      tc_fence_after();
      for (int i = 0; i < kAhead && i < n; ++i) {
        if (!(ok = arrived(g))) break;
        qk(NQT == 1 ? i : 0, g, NQT == 1);
        if (NQT == 2) qk(1, g, true);
        ++g;
      }
      for (int i = 0; ok && i < n; ++i) {
        const bool more = i + kAhead < n;
        const uint32_t gv = g++, gk = more ? g++ : 0;
        if (!(ok = pv(NQT == 1 ? i & 1 : 0, gv, i < kAhead, NQT == 1))) break;
        if (more) {
          if (!(ok = arrived(gk))) break;
          qk(NQT == 1 ? i & 1 : 0, gk, NQT == 1);
        }
        if (NQT == 2) {
          if (!(ok = pv(1, gv, i == 0, true))) break;
          if (more) qk(1, gk, true);
        }
      }
      if (!ok) break;
      commit(bar(B_OFINAL));
      ++n_piece;
    }
    __syncwarp();
    commit(bar(B_FINAL));
    mbar_wait(bar(B_FINAL), 0, kWaitLimitNs);
  } else if (warp >= W_SOFTMAX0) {
    // a stream's warps: HALVES for each lane quarter, 16 lanes each
    const int stream = (warp - W_SOFTMAX0) / kStreamWarps, quarter = warp & 3;
    const int hf = HALVES == 2 ? ((warp - W_SOFTMAX0) >> 2) & 1 : 0;
    const int cq = lane & 3;
    const uint32_t tS = tmem + ((uint32_t)(quarter * 32 + hf * 16) << 16) + stream * 128;
    const uint32_t tO = tS + 256;
    const float c = p.scale_log2;
    const uint64_t c2 = pk2(c, c);
    // written by every softmax warp with the same values
    uint64_t* see = reinterpret_cast<uint64_t*>(smem + OFF_SEE);
    uint32_t g = 0, n_t = 0, n_piece = 0;   // ring tiles and this stream's tiles used so far, pieces
    bool ok = true;
    while (ok && walk.next(p, &w)) {
      // ---- the query tiles: each warp loads an equal share of the shared-memory rows; rows of
      // missing tokens are zeros (NaN among them would never get a reference)
      const __nv_bfloat16* q_head = p.Q + ((long long)w.b * p.Hq + (long long)w.h * p.G) * p.T * kHeadDim;
      const int row0 = w.block * (NQT == 2 ? 2 * BM : BM);      // first row of the block
      const int ch = lane & 15;
      constexpr int kEach = NQT * MQ / (2 * kStreamWarps) / 2;   // 16-byte words of a lane
      uint4 v[kEach];
#pragma unroll
      for (int it = 0; it < kEach; ++it) {
        const int at = (warp - W_SOFTMAX0) * 2 * kEach + it * 2 + (lane >> 4), L = at & (MQ - 1);
        const int r = row0 + (at >> kQBits) * BM + 4 * (L & (kLanes - 1)) + (L >> (kQBits - 2));
        v[it] = make_uint4(0, 0, 0, 0);
        if (r < p.rows && (w.draft == p.T || r % p.T < w.draft))
          v[it] = *reinterpret_cast<const uint4*>(q_head + (long long)r * kHeadDim + ch * 8);
      }
#pragma unroll
      for (int it = 0; it < kEach; ++it) {
        const int at = (warp - W_SOFTMAX0) * 2 * kEach + it * 2 + (lane >> 4), L = at & (MQ - 1);
        *reinterpret_cast<uint4*>(smem + (at >> kQBits) * kQTile + (ch >> 3) * kQHalf + L * 128 +
                                  (((ch & 7) ^ (L & 7)) << 4)) = v[it];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_QREADY));

      // ---- this thread's rows: of the warp's 16 lanes, A (lane / 4) and B (+ 8)
      const int srow0 = row0 + (NQT == 2 ? stream * BM : 0);    // first row of this stream's tile
      const int srows = min(p.rows - srow0, BM);                // valid rows of it (can be <= 0)
      const int in_q = srows > quarter ? (srows - quarter + 3) >> 2 : 0;   // of this quarter
      const int groups = min(max(((in_q + 7) >> 3) - 2 * hf, 0), 2);      // of eight rows, this warp's
      const int rowA = 4 * (16 * hf + (lane >> 2)) + quarter, rowB = rowA + 32;     // within the tile
      const int tail0 = w.len / BN;                             // first tile with drafted or empty slots
      const bool tail = w.t0 + w.n > tail0;
      if (tail) {
        const Sees sv = tree_sees(p, w.b, w.draft, lane);
        see[lane] = sv.m0;
        see[lane + 32] = sv.m1;
        __syncwarp();
      }
      // per row: reference score, two partial sums
      float m[2];
      uint64_t l[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[k] = -INFINITY;
        l[k] = 0ull;
      }
      constexpr int step = NQT == 1 ? 2 : 1;
      for (int i = NQT == 1 ? stream : 0; i < w.n; i += step, ++n_t) {
        const int k0 = (w.t0 + i) * BN;             // first slot of the tile
        // V rows past the last slot: zero them before the product reads them
        const int slots = w.len + w.draft;
        if (k0 + BN > slots && (NQT == 1 || stream == 0)) {
          const uint32_t q = g + 2 * w.n - 1;      // the item's last tile is the piece's last load
          if (!(ok = wait(bar(B_FULL + q % NST), (q / NST) & 1))) break;
          unsigned char* v = smem + NQT * kQTile + (q % NST) * kKvBytes;
          for (int x = (slots - k0) * 16 + (hf * 4 + quarter) * 32 + lane; x < BN * 16; x += 32 * kStreamWarps)
            *reinterpret_cast<uint4*>(v + (x & 1) * kKvHalfBytes + (x >> 1) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        if (!(ok = wait(bar(B_SFULL + stream), n_t & 1))) break;
        tc_fence_after();
        // two halves of 64 slots; P of a half goes over S of the first one
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (groups > 0) {
            const uint32_t tSh = tS + half * 64, tP = tS + half * 32;
            // s[4j + e]: row A, slot k0 + 64 half + 8j + 2cq + e; s[4j + 2 + e]: row B
            uint32_t s[32];
            tmem_ld_16x256b_x8(tSh, s);
            tmem_wait_ld_of(s);
            auto S = [&](int gr, int j, int e) -> uint32_t& { return s[4 * j + 2 * gr + e]; };
            const int n0 = w.len - k0 - 64 * half;      // slots of the half that hold cached keys
            auto mask = [&] {
              if (n0 >= 64) return;
#pragma unroll
              for (int gr = 0; gr < 2; ++gr) {
                const uint64_t sees = see[(srow0 + rowA + 32 * gr) % p.T];
                uint64_t vis = n0 > 0 ? (sees << n0) | ((1ull << n0) - 1) : n0 > -64 ? sees >> -n0 : 0ull;
                vis >>= 2 * cq;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (!((vis >> (8 * j + e)) & 1)) S(gr, j, e) = __float_as_uint(-INFINITY);
              }
            };
            mask();
            if (HALVES == 1 && p.scores) {      // for the weight pass
#pragma unroll
              for (int gr = 0; gr < 2; ++gr) {
                const int r = rowA + 32 * gr;
                if (r >= p.rows) break;
                float* d = p.scores + (((long long)w.b * p.Hkv + w.h) * p.rows + r) * p.score_cap + k0 + 64 * half + 2 * cq;
#pragma unroll
                for (int j = 0; j < 8; ++j) *reinterpret_cast<uint2*>(d + 8 * j) = make_uint2(S(gr, j, 0), S(gr, j, 1));
              }
            }
            // The difference is taken before the scale: scores near the
            // reference keep their distance to it exactly, however large they
            // are. A row that has seen nothing yet keeps m = -inf: its p are 0.
            // pk[2j]: row A, pk[2j + 1]: row B (16x128b: lanes t / 4 and t / 4 + 8)
            uint32_t pk[16];
            uint64_t sum[2];
            float top = 0.f;
            auto exps = [&] {
#pragma unroll
              for (int gr = 0; gr < 2; ++gr) {
                sum[gr] = 0ull;
                if (groups > gr) {
                  const float n = m[gr] == -INFINITY ? 0.f : -m[gr];
                  const uint64_t n2 = pk2(n, n);
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    float x0, x1;
                    unpk2(mul2(add2(pk2(__uint_as_float(S(gr, j, 0)), __uint_as_float(S(gr, j, 1))), n2), c2), x0, x1);
                    x0 = fast_exp2(x0);
                    x1 = fast_exp2(x1);
                    top = max3(top, x0, x1);
                    sum[gr] = add2(sum[gr], pk2(x0, x1));
                    pk[2 * j + gr] = pack_bf16x2(x0, x1);
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 8; ++j) pk[2 * j + gr] = 0u;
                }
              }
            };
            // The first half has no reference yet. (With 640 threads the branch
            // costs the loop its registers: 157 us against 144 for 256 rows
            // over 131000 slots, 17.8 against 16.6 for 128 rows of 8 sequences
            // over 500; with 384 it saves 0.3 of 7.7 us for 37 slots.)
            const bool start = HALVES == 1 && i < step && half == 0;
            if (!start) exps();
            // Scores are taken relative to a reference of the row, its
            // largest score when the reference was last set: it is set again,
            // and O rescaled, only when a score passes it by 2^kRaise. P and
            // the sums have fp32's exponent range, so O / l is the same; the
            // test needs no exchange between the row's threads, and comes
            // after the exponentials, which are seldom done again.
            const bool unset = m[0] == -INFINITY || (groups > 1 && m[1] == -INFINITY);
            if (start || __any_sync(0xffffffffu, top > kTop || unset)) {
              if (!start) {      // the scores again, in place of their p
                tmem_ld_16x256b_x8(tSh, s);
                tmem_wait_ld_of(s);
                mask();
              }
              float f[2];
#pragma unroll
              for (int gr = 0; gr < 2; ++gr) {
                float x = -INFINITY;
                if (groups > gr) {
#pragma unroll
                  for (int j = 0; j < 8; ++j) x = max3(x, __uint_as_float(S(gr, j, 0)), __uint_as_float(S(gr, j, 1)));
                }
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                const bool r = (x - m[gr]) * c > kRaise;      // the row's own need: no other row shows in it
                f[gr] = r ? fast_exp2((m[gr] - x) * c) : 1.f;
                if (r) m[gr] = x;
                l[gr] = mul2(l[gr], pk2(f[gr], f[gr]));
              }
              // S complete implies the products of the stream's earlier tiles complete
              if (half == 1 && !(ok = wait(bar(B_PVHALF + stream), n_t & 1))) break;
              tc_fence_after();
              exps();
              if (i >= step || half == 1) {
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                  uint32_t o[16];
                  tmem_ld_16x256b_x4(tO + 32 * q, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f[(j >> 1) & 1]);
                  tmem_st_16x256b_x4(tO + 32 * q, o);
                }
              }
            }
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) l[gr] = add2(l[gr], sum[gr]);
            tmem_st_16x128b_x8(tP, pk);
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_PREADY + 2 * stream + half));
        }
        if (!ok) break;
      }
      if (!ok) break;
      g += 2 * w.n;
      if (warp == W_SOFTMAX0 && lane == 0 && !p.whole) {
        if (w.first) p.span[w.item].x = blockIdx.x;
        if (w.last) p.span[w.item].y = blockIdx.x;
      }
      // ---- the piece's result
      if (!(ok = wait(bar(B_OFINAL), n_piece & 1))) break;
      tc_fence_after();
      float sum[2];
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        float y;
        unpk2(l[gr], sum[gr], y);
        sum[gr] += y;
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
      }
      // With one query tile both streams hold parts of the same rows, O in
      // the same TMEM lanes: stream 1 hands over its references and sums, and
      // stream 0 joins the two.
      float f0[2], f1[2];
      float2* xchg = reinterpret_cast<float2*>(smem + OFF_XCHG) + quarter * 32 + 16 * hf + (lane >> 2);
      if (NQT == 1 && stream == 1) {
#pragma unroll
        for (int gr = 0; gr < 2; ++gr)
          if (cq == 0) xchg[8 * gr] = make_float2(m[gr], sum[gr]);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_XCHG + 2 * quarter + hf));
      } else if (NQT == 1) {
        if (!(ok = wait(bar(B_XCHG + 2 * quarter + hf), n_piece & 1))) break;
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          const float2 o = xchg[8 * gr];
          const float top = fmaxf(m[gr], o.x);
          f0[gr] = m[gr] == -INFINITY ? 0.f : fast_exp2((m[gr] - top) * c);
          f1[gr] = o.x == -INFINITY ? 0.f : fast_exp2((o.x - top) * c);
          m[gr] = top;
          sum[gr] = sum[gr] * f0[gr] + o.y * f1[gr];
        }
      }
      ++n_piece;
      if ((NQT == 2 || stream == 0) && groups > 0) {
        const long long out_row = ((long long)w.b * p.Hq + (long long)w.h * p.G) * p.T + srow0;
        const long long slot = ((long long)blockIdx.x + w.item) * NQT + (NQT == 2 ? stream : 0);
        const bool two = NQT == 1 && w.n > 1;      // stream 1 had a tile
        // a complete item is normalised here, rows of missing tokens are not written
        const bool wa = rowA < srows && (!w.complete || (srow0 + rowA) % p.T < w.draft);
        const bool wb = rowB < srows && (!w.complete || (srow0 + rowB) % p.T < w.draft);
        float ga = 1.f, gb = 1.f;
        if (w.complete) {
          ga = sum[0] > 0.f ? 1.f / sum[0] : 0.f;
          gb = sum[1] > 0.f ? 1.f / sum[1] : 0.f;
        }
        if (cq == 0) {
          auto keep = [&](int r, int gr) {
            if (!w.complete) {
              p.part_ml[slot * p.row_cap + r] = make_float2(m[gr], sum[gr]);
            } else {
              if (p.lse) p.lse[out_row + r] = m[gr] * p.scale + logf(sum[gr]);
              if (p.row_stat) p.row_stat[out_row + r] = make_float2(m[gr], 1.f / sum[gr]);
            }
          };
          if (wa) keep(rowA, 0);
          if (wb) keep(rowB, 1);
        }
        const float a0 = NQT == 1 ? f0[0] * ga : ga, b0 = NQT == 1 ? f0[1] * gb : gb;
        const float a1 = NQT == 1 ? f1[0] * ga : 0.f, b1 = NQT == 1 ? f1[1] * gb : 0.f;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t o[16], o1[16];
          tmem_ld_16x256b_x4(tO + 32 * q, o);
          if (two) tmem_ld_16x256b_x4(tO + 128 + 32 * q, o1);
          tmem_wait_ld();
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[j] = __uint_as_float(o[j]) * ((j & 2) ? b0 : a0);
            if (two) v[j] = fmaf(__uint_as_float(o1[j]), (j & 2) ? b1 : a1, v[j]);
          }
          if (w.complete) {
            __nv_bfloat16* oa = p.O + (out_row + rowA) * kHeadDim + 32 * q + 2 * cq;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (wa) *reinterpret_cast<uint32_t*>(oa + 8 * j) = pack_bf16x2(v[4 * j], v[4 * j + 1]);
              if (wb) *reinterpret_cast<uint32_t*>(oa + 32 * kHeadDim + 8 * j) = pack_bf16x2(v[4 * j + 2], v[4 * j + 3]);
            }
          } else {
            float* oa = p.part_o + (slot * p.row_cap + rowA) * kHeadDim + 32 * q + 2 * cq;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (wa) *reinterpret_cast<float2*>(oa + 8 * j) = make_float2(v[4 * j], v[4 * j + 1]);
              if (wb) *reinterpret_cast<float2*>(oa + 32 * kHeadDim + 8 * j) = make_float2(v[4 * j + 2], v[4 * j + 3]);
            }
          }
        }
      }
      tc_fence_before();
    }
  }

  // Every warp reports and exits; warp 1 frees TMEM once all have.
  __syncwarp();
  tc_fence_before();
  if (warp != W_MMA) {
    if (lane == 0) mbar_arrive(bar(B_TEARDOWN));
    return;
  }
  mbar_wait(bar(B_TEARDOWN), 0, kWaitLimitNs);
  __syncwarp();
  tc_fence_after();
  tmem_dealloc(tmem, kTmemCols);
}

struct Plan {
  int rows, wide, blocks, row_cap, score_cap;
  bool whole, scores;
  size_t o_bytes, ml_bytes, span_bytes, stat_bytes, score_bytes;
};
Plan make_plan(int B, int Hq, int Hkv, int T, int cap, bool want_weight) {
  Plan q;
  q.rows = Hq / Hkv * T;
  q.wide = q.rows > BM ? 2 : 1;
  q.blocks = ceil_div(q.rows, q.wide * BM);
  q.row_cap = q.rows < BM ? q.rows : BM;
  q.score_cap = ceil_div(cap, BN) * BN;
  q.whole = cap <= (B * (long long)Hkv * q.blocks >= kManyItems ? kWholeTilesMany : kWholeTiles) * BN;
  q.scores = want_weight && q.rows <= kMaxScoreRows;
  const size_t pieces = q.whole ? 0 : (size_t)B * Hkv * q.blocks + kMaxGrid;
  auto round = [](size_t n) { return (n + 255) / 256 * 256; };
  q.o_bytes = round(pieces * q.wide * q.row_cap * kHeadDim * sizeof(float));
  q.ml_bytes = round(pieces * q.wide * q.row_cap * sizeof(float2));
  q.span_bytes = q.whole ? 0 : round(sizeof(int2) * (size_t)B * Hkv * q.blocks);
  q.stat_bytes = want_weight ? round(sizeof(float2) * (size_t)B * Hq * T) : 0;
  q.score_bytes = q.scores ? sizeof(float) * (size_t)B * Hkv * q.rows * q.score_cap : 0;
  return q;
}

}  // namespace

int tree_max_drafts() { return kMaxDrafts; }
int tree_max_group() { return kMaxGroup; }

size_t tree_ws_bytes(int B, int Hq, int Hkv, int T, int cap, bool want_weight) {
  const Plan q = make_plan(B, Hq, Hkv, T, cap, want_weight);
  return 256 + q.o_bytes + q.ml_bytes + q.span_bytes + q.stat_bytes + q.score_bytes;
}

int launch_tree_attn(const void* Q, const void* K, const RowStrides& ks, const void* V, const RowStrides& vs, int B,
                     int Hq, int Hkv, int T, int cap, const int32_t* lengths, const int32_t* parents,
                     const int32_t* n_draft, float softmax_scale, void* O, float* lse, const float* weight,
                     float* weight_out, void* ws, unsigned int* status, cudaStream_t stream) {
  const Plan q = make_plan(B, Hq, Hkv, T, cap, weight_out != nullptr);
  EncodeTiledFn enc = tmap_encode_fn();
  if (!enc) return cuda_status(cudaErrorNotSupported);
  TreeMaps maps;
  if (!make_cache_map(enc, &maps.k, K, ks, B, Hkv, cap, BN) || !make_cache_map(enc, &maps.v, V, vs, B, Hkv, cap, BN))
    return DHSA_ERR_INVALID_ARG;
  static std::atomic<bool> done[3][64];
  int dev = 0, sms = 0;
  cudaError_t e = this_device(&dev, &sms);
  // Rows beyond 64 need both halves of the lanes of each quarter; up to 64,
  // warps for both would leave half of them without rows (98.9 against 92.8 us
  // for one token over 131071 slots). Beyond, a warp for each half beats one
  // for both: 305 against 320 us for 64 tokens with weights.
  const int halves = q.rows > 64 ? 2 : 1;
  auto* kernel = q.wide == 2 ? tree_attn_kernel<2, 2> : halves == 2 ? tree_attn_kernel<1, 2> : tree_attn_kernel<1, 1>;
  if (e == cudaSuccess) e = allow_smem(kernel, (int)kSmemAlloc, dev, done[q.wide + halves - 2]);
  if (e != cudaSuccess) return cuda_status(e);

  TreeParams p;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.lengths = lengths;
  p.parents = parents;
  p.n_draft = n_draft;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  char* at = static_cast<char*>(ws);
  p.part_o = reinterpret_cast<float*>(at);
  p.part_ml = reinterpret_cast<float2*>(at += q.o_bytes);
  p.span = reinterpret_cast<int2*>(at += q.ml_bytes);
  p.row_stat = reinterpret_cast<float2*>(at += q.span_bytes);
  p.scores = reinterpret_cast<float*>(at += q.stat_bytes);
  if (!weight_out) p.row_stat = nullptr;
  if (!q.scores) p.scores = nullptr;
  p.weight = weight;
  p.weight_out = weight_out;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.T = T;
  p.cap = cap;
  p.rows = q.rows;
  p.blocks = q.blocks;
  p.row_cap = q.row_cap;
  p.every = false;
  p.score_cap = q.score_cap;
  p.whole = q.whole;
  p.keep_k = weight_out && !q.scores;
  const long long most = (long long)B * Hkv * q.blocks * (q.whole ? 1 : ceil_div(cap, BN));   // the line's length at most
  p.grid = sms < kMaxGrid ? sms : kMaxGrid;
  if (most < p.grid) p.grid = (int)most;
  p.scale = softmax_scale;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.status = status;
  unsigned long long limit_ns;
  p.hold = 0;
  if (take_wait_test(1, &limit_ns))      // test hook: the first waits run out
    while (1ull << ++p.hold < limit_ns) {}
  kernel<<<p.grid, block_threads(halves), kSmemAlloc, stream>>>(maps, p);
  int st = launch_status();
  if (st == DHSA_OK && q.scores) {
    st = launch_tree_join_weights(p, stream);
  } else if (st == DHSA_OK && !q.whole) {
    st = launch_tree_join(p, stream);
  }
  if (st == DHSA_OK && weight_out && !q.scores) {
    p.whole = false;
    p.every = true;                   // weights without new tokens are passed on
    p.blocks = 1;                     // one walk over the keys for all rows of a head
    p.grid = sms < kMaxGrid ? sms : kMaxGrid;
    const long long tiles = (long long)B * Hkv * ceil_div(cap, kTileSlots);
    if (tiles < p.grid) p.grid = (int)tiles;
    CUtensorMap kmap;
    if (!make_cache_map(enc, &kmap, K, ks, B, Hkv, cap, kTileSlots)) return DHSA_ERR_INVALID_ARG;
    st = launch_tree_weight(kmap, p, stream);
  }
  return st;
}

}  // namespace dhsa
