// What follows the attention of tree_attn.cu: joins the pieces of rows that
// several CTAs shared, and, for few rows, the slots' weights.
//
// Both are a pass over data that mostly sits in L2, and short: what counts is
// the chain of dependent loads. So every row, and every block of slots, finds
// its row statistics for itself from the pieces (at most one per CTA), and
// where both are wanted they are one launch. Measured: 32 rows of 18 pieces
// each 3 us behind the attention, 2048 rows 5 us (19 MB of pieces); 256 rows of
// 32 sequences with the weights of 1.2M slots 8 us.
#include "tree.cuh"

namespace dhsa {
namespace {

// Where a row's pieces are: CTAs c0 .. c1 of its item, or one CTA that wrote
// the row itself.
struct RowPieces {
  int c0, c1, item, wide, tile, tr;
  __device__ __forceinline__ bool complete() const { return c0 == c1; }
  __device__ __forceinline__ long long at(const TreeParams& p, int c) const {
    return ((long long)(c + item) * wide + tile) * p.row_cap + tr;
  }
};
__device__ __forceinline__ RowPieces row_pieces(const TreeParams& p, int bh, int r) {
  RowPieces q;
  q.wide = p.rows > kTileRows ? 2 : 1;              // query tiles of a block
  q.item = bh * p.blocks + r / (q.wide * kTileRows);
  q.tile = r / kTileRows % q.wide;
  q.tr = r % kTileRows;
  const int2 span = p.whole ? make_int2(0, 0) : p.span[q.item];
  // (a CTA whose wait ran out leaves its span unwritten: the rows are wrong, and flagged, but stay in range)
  q.c0 = (int)min((unsigned)span.x, (unsigned)(p.grid - 1));
  q.c1 = max(q.c0, (int)min((unsigned)span.y, (unsigned)(p.grid - 1)));
  return q;
}

// by one warp: the pieces' common reference M and the row's denominator
// sum_i f_i l_i, f_i = exp(scale (m_i - M)); f (one per CTA) gets the factors
__device__ __forceinline__ float2 row_denominator(const TreeParams& p, const RowPieces& q, int lane, float* f) {
  float mx = -INFINITY;
  float2 first = make_float2(-INFINITY, 0.f);       // the lane's first piece; few rows have more
  if (q.c0 + lane <= q.c1) first = p.part_ml[q.at(p, q.c0 + lane)];
  mx = first.x;
  for (int c = q.c0 + 32 + lane; c <= q.c1; c += 32) mx = fmaxf(mx, p.part_ml[q.at(p, c)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float l = 0.f;
  for (int c = q.c0 + lane; c <= q.c1; c += 32) {
    const float2 ml = c == q.c0 + lane ? first : p.part_ml[q.at(p, c)];
    const float k = ml.x == -INFINITY ? 0.f : fast_exp2((ml.x - mx) * p.scale_log2);
    l += k * ml.y;
    f[c - q.c0] = k;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  return make_float2(mx, l);
}

// by one warp: O = sum_i f_i O_i / sum_i f_i l_i of one row, 16 bytes a lane
__device__ __forceinline__ void join_row(const TreeParams& p, int bh, int r, int lane, float* f) {
  const RowPieces q = row_pieces(p, bh, r);
  if (q.complete()) return;                          // one CTA had the whole item and wrote its rows
  const float2 ml = row_denominator(p, q, lane, f);
  __syncwarp();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* part = p.part_o + q.at(p, q.c0) * kHeadDim + 4 * lane;
  const long long step = (long long)q.wide * p.row_cap * kHeadDim;
  const int n = q.c1 - q.c0 + 1;
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const float k = f[i];
    const float4 v = *reinterpret_cast<const float4*>(part + i * step);
    o.x += k * v.x;
    o.y += k * v.y;
    o.z += k * v.z;
    o.w += k * v.w;
  }
  const long long row = (long long)bh * p.rows + r;
  const float g = ml.y > 0.f ? 1.f / ml.y : 0.f;
  *reinterpret_cast<uint2*>(p.O + row * kHeadDim + 4 * lane) =
      make_uint2(pack_bf16x2(o.x * g, o.y * g), pack_bf16x2(o.z * g, o.w * g));
  if (lane == 0) {
    if (p.lse) p.lse[row] = ml.x * p.scale + logf(ml.y);
    if (p.row_stat) p.row_stat[row] = make_float2(ml.x, 1.f / ml.y);
  }
}

// One block of one warp per row. (Blocks of four warps took 1 to 3 us more,
// and so did letting them start while the attention runs: they then crowd on
// the SMs that are free first.)
__global__ void __launch_bounds__(32) tree_join_kernel(const TreeParams p) {
  __shared__ float f[kMaxGrid];
  launch_dependents();
  const int r = (int)(blockIdx.x % (unsigned)p.rows), bh = (int)(blockIdx.x / (unsigned)p.rows);
  const SeqLen s = seq_len(p.lengths, p.n_draft, p.T, bh / p.Hkv, p.T, p.cap);
  wait_for_predecessors();       // before any return: no kernel of the chain ends before the one it follows
  if (r % p.T < s.draft) join_row(p, bh, r, threadIdx.x, f);
}

// Rows and slots in one launch: the first blocks join rows, a warp each; every
// other one adds the p of its head's rows (at most kMaxScoreRows) to 1024
// slots, from the scores that the attention kept: 8 bytes per slot and row
// instead of K's 256, and nothing to compute but the exponentials.
constexpr int kThreads = 256, kWarps = kThreads / 32, kSlotsEach = 4, kSlots = kThreads * kSlotsEach;
__global__ void __launch_bounds__(kThreads) tree_join_weights_kernel(const TreeParams p, unsigned row_blocks) {
  __shared__ float f[kWarps][kMaxGrid];
  __shared__ float2 stat[kMaxScoreRows];       // reference score, 1 / denominator (0: a missing token's row)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x < row_blocks) {
    const long long row = (long long)blockIdx.x * kWarps + warp;
    const int r = (int)(row % p.rows), bh = (int)(row / p.rows);
    const bool inside = bh < p.B * p.Hkv;
    const SeqLen s = seq_len(p.lengths, p.n_draft, p.T, inside ? bh / p.Hkv : 0, p.T, p.cap);
    wait_for_predecessors();
    if (inside && r % p.T < s.draft) join_row(p, bh, r, lane, f[warp]);
    return;
  }
  const unsigned parts = (unsigned)(p.cap + kSlots - 1) / kSlots, at = blockIdx.x - row_blocks;
  const int bh = (int)(at / parts), b = bh / p.Hkv;
  const SeqLen s = seq_len(p.lengths, p.n_draft, p.T, b, p.T, p.cap);
  const int block0 = (int)(at % parts) * kSlots, first = block0 + threadIdx.x;
  float old[kSlotsEach];
#pragma unroll
  for (int k = 0; k < kSlotsEach; ++k) {
    const int slot = first + k * kThreads;
    old[k] = slot < s.len ? p.weight[(long long)bh * p.cap + slot] : 0.f;
  }
  wait_for_predecessors();
  if (block0 >= s.len + s.draft) return;
  // Few rows are one query tile, so the head is one item; without drafted
  // tokens there was no item, and `span` has nothing for it. The chains of the
  // rows' loads run side by side.
  const int rows = s.draft > 0 ? p.rows : 0;
  const RowPieces q = rows ? row_pieces(p, bh, 0) : RowPieces{};
  if (q.complete()) {
    const int r = threadIdx.x;
    if (r < rows) stat[r] = r % p.T < s.draft ? p.row_stat[(long long)bh * p.rows + r] : make_float2(0.f, 0.f);
  } else {
    constexpr int kEach = kMaxScoreRows / kWarps;
    float mx[kEach], l[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      mx[i] = -INFINITY;
      l[i] = 0.f;
    }
    for (int c0 = q.c0; c0 <= q.c1; c0 += 32) {
      float2 ml[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = warp + i * kWarps;
        ml[i] = make_float2(-INFINITY, 0.f);
        if (c0 + lane <= q.c1 && r < rows) ml[i] = p.part_ml[q.at(p, c0 + lane) + r];
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        float top = fmaxf(mx[i], ml[i].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // a lane's sum so far is relative to the old reference
        const float keep = mx[i] == -INFINITY ? 0.f : fast_exp2((mx[i] - top) * p.scale_log2);
        const float add = ml[i].x == -INFINITY ? 0.f : fast_exp2((ml[i].x - top) * p.scale_log2);
        l[i] = l[i] * keep + add * ml[i].y;
        mx[i] = top;
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      const int r = warp + i * kWarps;
      if (lane == 0 && r < rows) stat[r] = r % p.T < s.draft ? make_float2(mx[i], 1.f / l[i]) : make_float2(0.f, 0.f);
    }
  }
  __syncthreads();
  float sum[kSlotsEach] = {0.f, 0.f, 0.f, 0.f};
  const float* scores = p.scores + (long long)bh * p.rows * p.score_cap + first;
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const float2 st = stat[r];
    float x[kSlotsEach];
#pragma unroll
    for (int k = 0; k < kSlotsEach; ++k)
      x[k] = first + k * kThreads < s.len + s.draft ? scores[(long long)r * p.score_cap + k * kThreads] : 0.f;
#pragma unroll
    for (int k = 0; k < kSlotsEach; ++k) {
      const float e = fast_exp2((x[k] - st.x) * p.scale_log2) * st.y;
      sum[k] += st.y == 0.f ? 0.f : e;         // a missing token's row: its scores can be anything
    }
  }
#pragma unroll
  for (int k = 0; k < kSlotsEach; ++k) {
    const int slot = first + k * kThreads;
    if (slot < s.len + s.draft) p.weight_out[(long long)bh * p.cap + slot] = old[k] + sum[k];
  }
}

}  // namespace

int launch_tree_join(const TreeParams& p, cudaStream_t stream) {
  return launch_after(tree_join_kernel, dim3((unsigned)((long long)p.B * p.Hkv * p.rows)), dim3(32), 0, stream, p);
}

int launch_tree_join_weights(const TreeParams& p, cudaStream_t stream) {
  const long long heads = (long long)p.B * p.Hkv;
  const unsigned row_blocks = p.whole ? 0u : (unsigned)((heads * p.rows + kWarps - 1) / kWarps);
  const unsigned slot_blocks = (unsigned)(heads * ceil_div(p.cap, kSlots));
  return launch_after(tree_join_weights_kernel, dim3(row_blocks + slot_blocks), dim3(kThreads), 0, stream, p, row_blocks);
}

}  // namespace dhsa
