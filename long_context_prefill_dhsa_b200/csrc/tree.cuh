// Shared by the kernels of the drafted-token attention (tree_attn.cu,
// tree_weight.cu): parameters, the split of the key tiles over the CTAs, the
// visibility of drafted tokens.
#pragma once
#include "cache.cuh"
#include "sm100_ptx.cuh"

namespace dhsa {

struct TreeParams {
  const __nv_bfloat16* Q;
  const int32_t *lengths, *parents, *n_draft;
  __nv_bfloat16* O;
  float* lse;
  float2* row_stat;         // per row: largest raw score and 1 / denominator, for the weight pass (null without)
  float* scores;            // [B * Hkv][rows][score_cap] raw scores for the weight pass, or null
  float* part_o;            // [piece][query tile][row_cap][128]
  int2* span;               // per item: the first and the last CTA that had a part of it
  float2* part_ml;          // [piece][query tile][row_cap]: reference score and sum
  const float* weight;
  float* weight_out;
  int B, Hq, Hkv, G, T, cap;
  int rows;                 // G * T
  int blocks;               // query blocks of a kv head that walk the keys
  int row_cap;              // rows of a query tile's partial
  int score_cap;            // cap rounded up to whole key tiles
  int grid;                 // CTAs that share the key tiles
  bool whole;               // items are not split: the line counts items instead of key tiles
  bool keep_k;              // K is read again after this kernel
  bool every;               // sequences without drafted tokens are walked too
  uint8_t hold;             // test hook, if not 0: no tile is loaded, and waits run out after 2^hold ns
  float scale, scale_log2;
  unsigned int* status;
};

namespace {

using namespace ptx;

constexpr int kMaxDrafts = 64;   // one bit of a 64-bit word each
constexpr int kMaxGroup = 64;    // query heads of one kv head
// Rows of a head up to which the attention keeps its scores (4 bytes per row
// and slot) for the slots' weights; with more rows the weights are computed
// again from K. Kept against computed again, us, 32/8 heads: one sequence of
// 131000 slots with 8, 16, 24, 32 rows 104, 119, 134, 150 against 168 to 171;
// 16 of 4000 to 8000 slots 83, 92, -, 118 against 163 to 166. Each further row
// adds about 2 us at 128K, so the two would meet near 42 rows. (33 to 42 take the
// longer way: the joining blocks have statistics for 32 rows, four a warp, and
// no limit between the two has been measured.)
constexpr int kMaxScoreRows = 32;
constexpr int kMaxGrid = 160;    // CTAs (one per SM) the workspace is sized for

constexpr int kTileSlots = 128;  // slots of a key tile
constexpr int kTileRows = 128;   // query rows of a query tile
constexpr uint32_t kTmemCols = 512;

// key tiles of each item of a sequence, and the item's length on the line
__device__ __forceinline__ int key_tiles(const TreeParams& p, const SeqLen& s) {
  return s.draft > 0 || p.every ? (s.len + s.draft + kTileSlots - 1) / kTileSlots : 0;
}
__device__ __forceinline__ int line_len(const TreeParams& p, const SeqLen& s) {
  const int n = key_tiles(p, s);
  return p.whole ? min(n, 1) : n;
}
__device__ __forceinline__ int line_len(const TreeParams& p, int b) {
  return line_len(p, seq_len(p.lengths, p.n_draft, p.T, b, p.T, p.cap));
}

// The line of key tiles, and how it is cut: sequence b's items start at
// `base`, and the CTA has [start, end).
//
// With fewer items than CTAs each item gets a whole number of CTAs in
// proportion to its tiles (`each` of them in sequence b, the first being CTA
// `first`), so that no CTA has parts of two: such a CTA would drain one item
// and fill its pipeline again for the next, about as long as five tiles (trees
// of 32 over 8 items of 8K slots: 48 us by items, 58 in equal shares). With
// more items the line is cut into equal shares.
// (At most 2^31 cached slots and 32 query blocks: the line is shorter than 2^30.)
struct Line {
  int start, end, base, b;
};

// start of share c of a line cut into `grid` equal shares: total c / grid
__device__ __forceinline__ int share_start(int total, int grid, int c) {
  return total / grid * c + total % grid * c / grid;
}
// CTAs that each item of a sequence with n tiles gets when the line is cut by items
__device__ __forceinline__ int item_ctas(const TreeParams& p, int n, int total) {
  return n ? max(1, min(n, (int)((unsigned)p.grid * (unsigned)n / (unsigned)total))) : 0;
}

// by one warp: the share of CTA c, with the sequence it starts in and that
// sequence's place. A line cut into equal shares is at least as long as there
// are CTAs, so no share of it is empty: shorter ones, and those with fewer
// items than CTAs, are cut by items (unless small items would take more CTAs
// than there are).
__device__ __forceinline__ Line find_share(const TreeParams& p, int c, int lane) {
  const int per = p.Hkv * p.blocks;
  const int n0 = lane < p.B ? line_len(p, lane) : 0;
  auto len_of = [&](int b0) { return b0 == 0 ? n0 : b0 + lane < p.B ? line_len(p, b0 + lane) : 0; };
  int sum = 0, some = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int n = len_of(b0);
    sum += n;
    some += n > 0;
  }
  const int total = per * __reduce_add_sync(0xffffffffu, sum);
  some = __reduce_add_sync(0xffffffffu, some);
  Line L{0, 0, 0, 0};
  if (total == 0) return L;
  bool by_item = (long long)some * per <= p.grid && !p.whole;
  if (by_item) {
    int ctas = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) ctas += item_ctas(p, len_of(b0), total);
    by_item = per * __reduce_add_sync(0xffffffffu, ctas) <= p.grid;
  }
  if (!by_item) {
    L.start = share_start(total, p.grid, c);
    L.end = share_start(total, p.grid, c + 1);
  }
  // the sequence that holds the share's start, or, by items, CTA c
  const int want = by_item ? c : L.start;
  int run = 0, run_base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B && run <= want; b0 += 32) {
    const int n = len_of(b0), k = by_item ? item_ctas(p, n, total) : n;
    int inc = k, inc_n = n;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o), vn = __shfl_up_sync(0xffffffffu, inc_n, o);
      if (lane >= o) {
        inc += v;
        inc_n += vn;
      }
    }
    const int from = run + (inc - k) * per, to = run + inc * per;
    const uint32_t hit = __ballot_sync(0xffffffffu, from <= want && want < to);
    if (hit) {
      const int src = __ffs(hit) - 1;
      L.b = b0 + src;
      L.base = run_base + __shfl_sync(0xffffffffu, inc_n - n, src) * per;
      if (by_item) {
        const int rel = c - __shfl_sync(0xffffffffu, from, src), each = __shfl_sync(0xffffffffu, k, src);
        const int nt = __shfl_sync(0xffffffffu, n, src), item = rel / each, part = rel % each;
        L.start = L.base + item * nt + share_start(nt, each, part);
        L.end = L.base + item * nt + share_start(nt, each, part + 1);
      }
      break;
    }
    run += __shfl_sync(0xffffffffu, inc, 31) * per;
    run_base += __shfl_sync(0xffffffffu, inc_n, 31) * per;
  }
  return L;
}

struct Piece {
  int b, h, block;
  int t0, n;            // key tiles t0 .. t0 + n - 1 of the item
  bool first, complete; // they begin the item; they are all of its tiles
  bool last;            // they end it
  int len, draft;
  int item;
};

// walks a CTA's share; every role does so on its own
struct Pieces {
  int pos, end, base;
  int b;
  __device__ __forceinline__ bool next(const TreeParams& p, Piece* o) {
    if (pos >= end) return false;
    const int per = p.Hkv * p.blocks;
    SeqLen s;
    int nt;
    for (;; ++b) {      // pos < end: a sequence with tiles follows
      s = seq_len(p.lengths, p.n_draft, p.T, b, p.T, p.cap);
      nt = line_len(p, s);
      if (pos < base + nt * per) break;
      base += nt * per;
    }
    const unsigned rel = (unsigned)(pos - base);
    const unsigned in_b = rel / (unsigned)nt;
    o->b = b;
    o->h = in_b / p.blocks;
    o->block = in_b % p.blocks;
    o->t0 = rel % (unsigned)nt;
    const int n = min(nt - o->t0, end - pos);
    o->first = o->t0 == 0;
    o->last = o->t0 + n == nt;
    o->complete = n == nt;
    o->n = p.whole ? key_tiles(p, s) : n;
    o->len = s.len;
    o->draft = s.draft;
    o->item = (b * p.Hkv + o->h) * p.blocks + o->block;
    pos += n;
    return true;
  }
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// pairs of fp32 in one 64-bit register, for the packed f32x2 operations
__device__ __forceinline__ uint64_t pk2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpk2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The drafted tokens each token sees, one bit each, by pointer doubling over
// the parents: lane l holds tokens l and l + 32.
struct Sees {
  uint64_t m0, m1;
  __device__ __forceinline__ uint64_t of(int t) const {   // all lanes, t in 0 .. 63
    const uint64_t a = __shfl_sync(0xffffffffu, m0, t & 31), c = __shfl_sync(0xffffffffu, m1, t & 31);
    return t < 32 ? a : c;
  }
};
__device__ __forceinline__ Sees tree_sees(const TreeParams& p, int b, int draft, int lane) {
  Sees s;
  const int t0 = lane, t1 = lane + 32;
  if (!p.parents) {
    s.m0 = t0 < draft ? (2ull << t0) - 1 : 0;
    s.m1 = t1 < draft ? (t1 == 63 ? ~0ull : (2ull << t1) - 1) : 0;
    return s;
  }
  int p0 = t0 < draft ? p.parents[b * p.T + t0] : -1, p1 = t1 < draft ? p.parents[b * p.T + t1] : -1;
  if (p0 < -1 || p0 >= t0 || p1 < -1 || p1 >= t1) {
    // a token without a usable parent hangs on the context
    if (p0 < -1 || p0 >= t0) p0 = -1;
    if (p1 < -1 || p1 >= t1) p1 = -1;
    raise_device_flag(p.status, DHSA_DEVFLAG_BAD_TREE);
  }
  s.m0 = t0 < draft ? 1ull << t0 : 0;
  s.m1 = t1 < draft ? 1ull << t1 : 0;
  while (__any_sync(0xffffffffu, p0 >= 0 || p1 >= 0)) {   // at most six rounds
    const Sees old = s;
    const int q0 = p0, q1 = p1;
    auto up = [&](int at) {
      const int a = __shfl_sync(0xffffffffu, q0, at & 31), c = __shfl_sync(0xffffffffu, q1, at & 31);
      return at < 32 ? a : c;
    };
    const int a0 = max(q0, 0), a1 = max(q1, 0);
    const uint64_t v0 = old.of(a0), v1 = old.of(a1);
    const int u0 = up(a0), u1 = up(a1);
    if (q0 >= 0) {
      s.m0 |= v0;
      p0 = u0;
    }
    if (q1 >= 0) {
      s.m1 |= v1;
      p1 = u1;
    }
  }
  return s;
}

// As in attn_fwd.cu: the lanes that wait together poll in lockstep and give up together.
struct Waits {
  volatile int* abort;      // [1]: the limit in ns
  unsigned int* status;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_test_wait(bar, parity)) return true;
    if (*abort) return false;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((it & 15u) == 0u && globaltimer_ns() - t0 > (unsigned)abort[1]) break;
    }
    if (mbar_test_wait(bar, parity)) return true;
    *abort = 1;
    raise_device_flag(status, DHSA_DEVFLAG_WAIT_TIMEOUT);
    return false;
  }
};

}  // namespace
}  // namespace dhsa
