// Eviction from a key/value cache by accumulated attention weight, and the
// commit of accepted drafts (the same update with room for every candidate).
//
// Each (sequence, kv head) keeps the m candidates that rank first: the held
// ones by slot, then the others by (weight descending, slot ascending). The
// rank is a 32-bit key whose unsigned order is that of the weights; held slots
// take the largest key, slots that are no candidates the key 0. The m-th
// largest key is found by a radix search (four 8-bit digits from the top, one
// histogram each); among equal keys the first slots win.
//
// The kept rows must end in slots 0 .. m-1, and the order of slots carries no
// meaning, so only as many rows move as there are unkept slots below m: the
// i-th such hole takes the i-th kept row from m on. Sources lie at m or
// above and destinations below, so the moves commute and need no order.
//
// One thread-block cluster per (sequence, head): its blocks split the slots,
// hold the keys in shared memory, and read each other's histograms and
// counts through distributed shared memory, so the whole update is one
// launch (two when few heads have many rows to move). Bound: 8 bytes (weight,
// position) per slot and 1 KB per moved row against HBM; for small caches the chain of four histogram rounds, one round
// of counts and their barriers. Measured: 8 heads of 131072 slots to 8192, 42.5
// us, 27 of them ranking (about 6 us until the keys are there, 3 a round, 10
// for counts and lists) and 12 moving 61K rows (63 MB at 5.3 TB/s).
#include <cooperative_groups.h>

#include <type_traits>

#include "cache.cuh"
#include "sm100_ptx.cuh"

namespace cg = cooperative_groups;

namespace dhsa {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 256;
constexpr int kParts = kEvThreads / kBins;
constexpr int kRounds = 4;
constexpr int kSplitMoves = 256;           // moves per block from which a second kernel does them
constexpr int kMaxCluster = 16;           // above 8 the launch asks for the non-portable size
constexpr int kLargeClusters = 14;        // clusters of 16 that the GPU runs at a time
constexpr int kBatch = 4;                 // slots whose weight and position a thread loads at a time
// Keys held in shared memory. A block with more slots than that derives keys
// again from the weights, and takes as long whether it holds 26K or 48K of them
// (4 heads of 1M slots: 205 us); with 26K two blocks fit an SM, and the clusters
// of 8 heads run at one time: 269 us against 419.
constexpr int kKeysPerBlock = 48 * 1024;
constexpr int kKeysOfMore = 26 * 1024;
constexpr int kSlotsPerBlock = 8192;      // slots a block of a cluster is given before another one joins

struct EvictParams {
  __nv_bfloat16 *K, *V;
  RowStrides ks, vs;
  const float* weight;
  const int32_t* pos;
  const int32_t *lengths, *n_draft, *next_pos;
  const int64_t* accept;
  float* weight_out;
  int32_t *pos_out, *lengths_out, *index;
  int32_t* lists;          // [B * Hkv][cap]: holes in the first half, their sources in the second
  uint32_t* moves;         // [B * Hkv] rows that move, when a second kernel moves them (else null)
  int B, Hkv, cap, keep, sinks, recent, index_cols, max_draft, keys_held;
  unsigned int* status;
};

// unsigned order = order of the floats, NaN lowest, -0 equal to +0; at least 1
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 1u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// counts of one range of slots: keys above the cut and equal to it, in slots
// below m and from m on
struct Counts {
  uint32_t gt_low, eq_low, gt_high, eq_high;
};

struct EvictShared {
  uint32_t hist[kRounds][kBins];
  uint32_t part[kParts][kBins];
  uint32_t warp_sum[kBins / 32];
  uint32_t pick_bin, pick_above, pick_all;
  Counts warp_count[kEvWarps];
  Counts total;              // this block's, read by the cluster
};

// what a range keeps, given how many equal keys before it stay
struct Kept {
  uint32_t low, high;
};
__device__ __forceinline__ Kept kept_of(const Counts& c, uint32_t eq_before, uint32_t ties) {
  const uint32_t left = ties > eq_before ? ties - eq_before : 0u;
  const uint32_t el = min(left, c.eq_low), eh = min(left - el, c.eq_high);
  return Kept{c.gt_low + el, c.gt_high + eh};
}
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {     // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The moves first, first + stride, ... of a head, by one warp: 16 lanes carry
// a slot's K row, 16 its V row. Sources and destinations are apart, so the
// moves need no order.
__device__ __forceinline__ void move_rows(const EvictParams& p, int b, int h, int bh, int lane, uint32_t moves,
                                          uint32_t first, uint32_t stride) {
  const long long row = (long long)bh * p.cap;
  const float* w_in = p.weight + row;
  const int32_t* pos_in = p.pos + row;
  float* w_out = p.weight_out + row;
  int32_t* pos_out = p.pos_out + row;
  int32_t* idx_row = p.index ? p.index + (long long)bh * p.index_cols : nullptr;
  const int32_t *hole_list = p.lists + row, *src_list = hole_list + p.cap / 2;
  const bool is_v = lane >= 16;
  __nv_bfloat16* base = is_v ? p.V + b * p.vs.b + h * p.vs.h : p.K + b * p.ks.b + h * p.ks.h;
  const long long rs = is_v ? p.vs.r : p.ks.r;
  base += (lane & 15) * 8;
  constexpr int kInFlight = 4;
  // lane l of a warp holds the l-th of its next 32 moves
  for (uint32_t r0 = first; r0 < moves; r0 += 32 * stride) {
    const uint32_t at = r0 + lane * stride;
    const int my_dst = at < moves ? hole_list[at] : -1, my_from = at < moves ? src_list[at] : 0;
    if (my_dst >= 0) {
      w_out[my_dst] = w_in[my_from];
      pos_out[my_dst] = pos_in[my_from];
      if (idx_row) idx_row[my_dst] = my_from;
    }
    const int n = __popc(__ballot_sync(0xffffffffu, my_dst >= 0));
    for (int k0 = 0; k0 < n; k0 += kInFlight) {
      uint4 x[kInFlight];
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int from = __shfl_sync(0xffffffffu, my_from, (k0 + k) & 31);
        if (k0 + k < n) x[k] = *reinterpret_cast<const uint4*>(base + from * rs);
      }
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int dst = __shfl_sync(0xffffffffu, my_dst, (k0 + k) & 31);
        if (k0 + k < n) *reinterpret_cast<uint4*>(base + dst * rs) = x[k];
      }
    }
  }
}

// SPLIT: the rows are moved by the next kernel
template <bool SPLIT>
__global__ void __launch_bounds__(kEvThreads, 2) evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) unsigned char ev_smem[];
  EvictShared& sh = *reinterpret_cast<EvictShared*>(ev_smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ev_smem + sizeof(EvictShared));
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int bh = blockIdx.x / C;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const SeqLen sl = seq_len(p.lengths, p.n_draft, 0, b, p.max_draft, p.cap);
  uint64_t bits = p.accept ? (uint64_t)p.accept[b] : ~0ull;
  bits &= sl.draft >= 64 ? ~0ull : (1ull << sl.draft) - 1;
  const int n_cand = sl.len + __popcll(bits), n_all = sl.len + sl.draft;
  const int m = min(p.keep, n_cand);
  if (sl.bad && rank == 0 && tid == 0) raise_device_flag(p.status, DHSA_DEVFLAG_BAD_CACHE);
  if (rank == 0 && h == 0 && tid == 0) p.lengths_out[b] = m;

  const long long row = (long long)bh * p.cap;
  const float* w_in = p.weight + row;
  const int32_t* pos_in = p.pos + row;
  const long long held_from = p.next_pos ? (long long)p.next_pos[b] - p.recent : (long long)INT32_MAX + 1;

  // this block's slots, and each warp's contiguous share of them
  const int per_warp = ceil_div(ceil_div(n_all, C * kEvWarps), 32) * 32;
  const int blk0 = rank * per_warp * kEvWarps;
  const int w0 = blk0 + warp * per_warp, w1 = min(w0 + per_warp, n_all);

  auto is_cand = [&](int s) { return s < sl.len || ((bits >> (s - sl.len)) & 1ull); };
  auto key_from = [&](int s, float w, int q) -> uint32_t {
    return !is_cand(s) ? 0u : (q < p.sinks || q >= held_from) ? 0xFFFFFFFFu : weight_key(w);
  };
  // What stays where it is, and the index of it: written for every slot below
  // m as it is first read; the holes among them are written again at the end.
  int32_t* idx_row = p.index ? p.index + (long long)bh * p.index_cols : nullptr;
  float* w_out = p.weight_out + row;
  int32_t* pos_out = p.pos_out + row;
  const bool copy_w = w_out != w_in, copy_pos = pos_out != pos_in;
  auto keep_in_place = [&](int s, float w, int q) {
    if (copy_w) w_out[s] = w;
    if (copy_pos) pos_out[s] = q;
    if (idx_row) idx_row[s] = s;
  };

  const bool all = m == n_cand;            // every candidate stays: no ranking
  uint32_t cut = 0;                        // the m-th largest key
  uint32_t ties = 0;                       // how many of the slots with that key stay
  // a block whose slots all have their key in shared memory has loops of its own
  const bool held = per_warp * kEvWarps <= p.keys_held;
  auto key_of = [&](auto in_shared, int s) -> uint32_t {
    if constexpr (in_shared.value) return keys[s - blk0];
    return s - blk0 < p.keys_held ? keys[s - blk0] : key_from(s, w_in[s], pos_in[s]);
  };
  auto with_keys = [&](auto f) {
    if (held) f(std::true_type{});
    else f(std::false_type{});
  };
  if (!all) {
    for (int i = tid; i < kRounds * kBins; i += kEvThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    for (int s0 = w0; s0 < w1; s0 += 32 * kBatch) {
      float w[kBatch];
      int q[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int s = s0 + 32 * u + lane;
        if (s < w1) {
          w[u] = w_in[s];
          q[u] = pos_in[s];
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int s = s0 + 32 * u + lane;
        if (s >= w1) break;
        const uint32_t k = key_from(s, w[u], q[u]);
        if (s - blk0 < p.keys_held) keys[s - blk0] = k;
        atomicAdd(&sh.hist[0][k >> 24], 1u);
        if (s < m) keep_in_place(s, w[u], q[u]);
      }
    }
    uint32_t left = (uint32_t)m;
#pragma unroll 1
    for (int r = 0; r < kRounds; ++r) {
      const int shift = 24 - 8 * r;
      if (r > 0)
        with_keys([&](auto in_shared) {
#pragma unroll 4
          for (int s = w0 + lane; s < w1; s += 32) {       // the lane's own keys
            const uint32_t k = key_of(in_shared, s);
            if ((k ^ cut) >> (shift + 8) == 0) atomicAdd(&sh.hist[r][(k >> shift) & 255u], 1u);
          }
        });
      cluster.sync();
      // the cluster's histogram: kParts threads per bin add up every kParts-th block's
      {
        uint32_t v = 0;
        const int bin = tid & 255;
#pragma unroll
        for (int i = 0; i < kMaxCluster / kParts; ++i) {       // all in flight at once
          const int c = (tid >> 8) + i * kParts;
          if (c < C) v += cluster.map_shared_rank(&sh.hist[r][0], c)[bin];
        }
        sh.part[tid >> 8][bin] = v;
      }
      __syncthreads();
      uint32_t n = 0, inc = 0;
      const int bin = kBins - 1 - tid;          // from the top
      if (tid < kBins) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) n += sh.part[i][bin];
        inc = warp_scan(n, lane);
        if (lane == 31) sh.warp_sum[warp] = inc;
      }
      __syncthreads();
      if (tid < kBins) {
        uint32_t before = inc - n;
#pragma unroll
        for (int i = 0; i < kBins / 32; ++i) before += i < warp ? sh.warp_sum[i] : 0u;
        if (before < left && left <= before + n) {       // exactly one bin
          sh.pick_bin = bin;
          sh.pick_above = before;
          sh.pick_all = left == before + n;
        }
      }
      __syncthreads();
      cut |= sh.pick_bin << shift;
      left -= sh.pick_above;
      if (sh.pick_all && cut != 0) {      // the whole bin stays: the cut lies right below it
        cut -= 1;
        left = 0;
        break;
      }
    }
    ties = left;
  }

  // counts of the warp's slots, then of every range before them
  Counts mine{0, 0, 0, 0};
  auto count = [&](int s, bool gt, bool eq) {
    const bool low = s < m;
    mine.gt_low += gt && low;
    mine.gt_high += gt && !low;
    mine.eq_low += eq && low;
    mine.eq_high += eq && !low;
  };
  if (all) {
    for (int s = w0 + lane; s < w1; s += 32) count(s, is_cand(s), false);
  } else {
    with_keys([&](auto in_shared) {
#pragma unroll 4
      for (int s = w0 + lane; s < w1; s += 32) {
        const uint32_t k = key_of(in_shared, s);
        count(s, k > cut, k == cut);
      }
    });
  }
  mine.gt_low = __reduce_add_sync(0xffffffffu, mine.gt_low);
  mine.gt_high = __reduce_add_sync(0xffffffffu, mine.gt_high);
  mine.eq_low = __reduce_add_sync(0xffffffffu, mine.eq_low);
  mine.eq_high = __reduce_add_sync(0xffffffffu, mine.eq_high);
  if (lane == 0) sh.warp_count[warp] = mine;
  __syncthreads();
  Counts wc{0, 0, 0, 0};                        // lane l: warp l's
  if (lane < kEvWarps) wc = sh.warp_count[lane];
  if (warp == 0) {
    Counts t;
    t.gt_low = __reduce_add_sync(0xffffffffu, wc.gt_low);
    t.gt_high = __reduce_add_sync(0xffffffffu, wc.gt_high);
    t.eq_low = __reduce_add_sync(0xffffffffu, wc.eq_low);
    t.eq_high = __reduce_add_sync(0xffffffffu, wc.eq_high);
    if (lane == 0) sh.total = t;
  }
  cluster.sync();
  Counts bc{0, 0, 0, 0};                        // lane c: block c's
  if (lane < C) bc = *cluster.map_shared_rank(&sh.total, lane);
  auto first = [&](uint32_t v, int n) { return __reduce_add_sync(0xffffffffu, lane < n ? v : 0u); };
  const uint32_t b_eq = bc.eq_low + bc.eq_high, w_eq = wc.eq_low + wc.eq_high;
  const Kept bk = kept_of(bc, warp_scan(b_eq, lane) - b_eq, ties);
  const uint32_t eq_block = first(b_eq, rank);
  const Kept wk = kept_of(wc, eq_block + warp_scan(w_eq, lane) - w_eq, ties);
  const uint32_t moves = first(bk.high, 32);    // kept slots from m on
  uint32_t tie_run = eq_block + first(w_eq, warp);
  uint32_t hole_at = (uint32_t)min(w0, m) - (first(bk.low, rank) + first(wk.low, warp));
  uint32_t src_at = first(bk.high, rank) + first(wk.high, warp);

  const uint32_t lt = (1u << lane) - 1;
  // the lists: for 32 consecutive slots of the warp at a time, in order
  int32_t* hole_list = p.lists + row;
  int32_t* src_list = hole_list + p.cap / 2;   // min(m, n_all - m) <= cap / 2 rows move
  auto list = [&](int s, bool yes) {
    const bool hole = s < m && s < w1 && !yes, src = s >= m && yes;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), sb = __ballot_sync(0xffffffffu, src);
    if (hole) hole_list[hole_at + __popc(hb & lt)] = s;
    if (src) src_list[src_at + __popc(sb & lt)] = s;
    hole_at += __popc(hb);
    src_at += __popc(sb);
  };
  if (all) {
    for (int s0 = w0; s0 < w1; s0 += 32) list(s0 + lane, s0 + lane < w1 && is_cand(s0 + lane));
  } else {
    with_keys([&](auto in_shared) {
#pragma unroll 4
      for (int s0 = w0; s0 < w1; s0 += 32) {
        const int s = s0 + lane;
        const uint32_t k = s < w1 ? key_of(in_shared, s) : 0u;
        const uint32_t eq = __ballot_sync(0xffffffffu, s < w1 && k == cut);
        list(s, s < w1 && (k > cut || (k == cut && tie_run + __popc(eq & lt) < ties)));
        tie_run += __popc(eq);
      }
    });
  }
  if (all && (copy_w || copy_pos || idx_row)) {
    for (int s0 = rank * kEvThreads + tid; s0 < m; s0 += C * kEvThreads * kBatch) {
      float w[kBatch];
      int q[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int s = s0 + u * C * kEvThreads;
        if (s < m) {
          w[u] = w_in[s];
          q[u] = pos_in[s];
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int s = s0 + u * C * kEvThreads;
        if (s < m) keep_in_place(s, w[u], q[u]);
      }
    }
  }
  if (idx_row)
    for (int s = m + rank * kEvThreads + tid; s < p.index_cols; s += C * kEvThreads) idx_row[s] = -1;
  // the cluster's lists are complete, and nobody reads a weight or position
  // to rank it any more
  cluster.sync();
  if (SPLIT) {
    if (rank == 0 && tid == 0) p.moves[bh] = moves;
  } else {
    move_rows(p, b, h, bh, lane, moves, rank * kEvWarps + warp, C * kEvWarps);
  }
}

// The rows of few heads, moved by the whole GPU.
__global__ void __launch_bounds__(kEvThreads, 2) evict_move_kernel(const EvictParams p, int blocks) {
  const int bh = blockIdx.x / blocks, part = blockIdx.x % blocks;
  ptx::wait_for_predecessors();
  move_rows(p, bh / p.Hkv, bh % p.Hkv, bh, threadIdx.x & 31, p.moves[bh], part * kEvWarps + (threadIdx.x >> 5),
            blocks * kEvWarps);
}

// More blocks per head shorten the loops over its slots and lengthen the
// rounds between them: 8 heads of 131072 slots take 49.7 us with 8, 44.9 with
// 10 and 43.6 with 16; 256 heads of 4112 slots 16.1 us with one block and 23.5
// with two. Of clusters of 16, 14 run at a time: 12 heads of 131072 slots take
// 47.3 us with 16 and 53.3 with 8, 16 heads 78 and 65. (The capacity decides,
// as the lengths are not known on the host: 8 heads with 8208 slots in use take
// 20.5 us in a cache of 131136 slots and 13.3 in one of 8208.)
int cluster_size(int cap, int heads) {
  int c = 1;
  while (c < kMaxCluster && (long long)c * kSlotsPerBlock < cap && (c < 8 || heads <= kLargeClusters)) c *= 2;
  return c;
}

}  // namespace

// the lists, and each head's number of moves
size_t evict_ws_bytes(int B, int Hkv, int cap) { return sizeof(int32_t) * (size_t)B * Hkv * ((size_t)cap + 1); }
int evict_max_drafts() { return 64; }

int launch_evict(void* K, const RowStrides& ks, void* V, const RowStrides& vs, const float* weight,
                 const int32_t* pos, int B, int Hkv, int cap, const int32_t* lengths, const int32_t* n_draft,
                 const int64_t* accept, int keep, int sinks, int recent, const int32_t* next_pos, float* weight_out,
                 int32_t* pos_out, int32_t* lengths_out, int32_t* index, void* ws, unsigned int* status,
                 cudaStream_t stream) {
  EvictParams p;
  p.K = static_cast<__nv_bfloat16*>(K);
  p.V = static_cast<__nv_bfloat16*>(V);
  p.ks = ks;
  p.vs = vs;
  p.weight = weight;
  p.pos = pos;
  p.lengths = lengths;
  p.n_draft = n_draft;
  p.next_pos = next_pos;
  p.accept = accept;
  p.weight_out = weight_out;
  p.pos_out = pos_out;
  p.lengths_out = lengths_out;
  p.index = index;
  p.lists = static_cast<int32_t*>(ws);
  p.B = B;
  p.Hkv = Hkv;
  p.cap = cap;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.index_cols = keep < cap ? keep : cap;
  p.max_draft = evict_max_drafts();
  p.status = status;
  const int C = cluster_size(cap, B * Hkv);
  const int span = ceil_div(cap, C * kEvThreads) * kEvThreads;   // slots of one block at most
  p.keys_held = span <= kKeysPerBlock ? span : kKeysOfMore;
  const size_t smem = sizeof(EvictShared) + 4u * (size_t)p.keys_held;
  static std::atomic<bool> done[2][64];
  int dev = 0, sms = 0;
  cudaError_t e = this_device(&dev, &sms);
  // When the clusters leave much of the GPU idle (8 of 16 blocks do, too: 7
  // places hold one) and there can be many moves, a second kernel moves the
  // rows, on all of it: 100000 of 300000 slots of one head 53 us against 118, 8
  // heads of 131072 to 8192 42.5 against 44.1, 96 heads of 4096 to 2048 37.3
  // against 38.0; but 128 heads of 4096 44.9 against 42.1, 10 heads of 131072
  // 51.0 against 47.2, and up to 128 moves a head take 12.3 either way.
  const int heads = B * Hkv, most = keep < cap - keep ? keep : cap - keep;
  const bool split = heads * C <= (C == kMaxCluster ? sms : 2 * sms / 3) && most >= kSplitMoves * C;
  p.moves = split ? reinterpret_cast<uint32_t*>(p.lists + (size_t)heads * cap) : nullptr;
  auto* kernel = split ? evict_kernel<true> : evict_kernel<false>;
  if (e == cudaSuccess && !done[split][dev])
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = allow_smem(kernel, (int)(sizeof(EvictShared) + 4u * (size_t)kKeysPerBlock), dev, done[split]);
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * Hkv * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess || !split) return cuda_status(e);
  const int blocks = ceil_div(2 * sms, heads);
  return launch_after(evict_move_kernel, dim3((unsigned)(heads * blocks)), dim3(kEvThreads), 0, stream, p, blocks);
}

}  // namespace dhsa
