// Attention of new tokens over the paged key-value cache for gfx950.
//
// What is computed, per query row (token t, head h; key-value head h / group):
//   out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j) over the keys j the row sees,
// in one pass over the keys with a running maximum m and sum l (exponentials in base 2, log2 e and the
// key scale folded into the factor c):  s_j = q . k_j,  m' = max(m, s),  l <- l 2^{(m - m') c} + sum 2^{(s - m') c},
// O <- O 2^{(m - m') c} + sum 2^{(s - m') c} v_j,  out = O / l * v_scale,  lse = (m c + log2 l) ln 2.
// m, l, O and the scores are fp32.  The factor by which old values are scaled down is applied only when
// the maximum grows by more than 2^8 (kLazy): until then probabilities are up to 2^8 times what they would be.
// Beside an E4M3 cache they are held 2^7 times larger (kLift; l, O and m c in the same scale): at most 2^15, within
// fp16's 65504, with a row's sum of at least 2^7.  fp16's smallest step, 2^-24, then takes at most 2^-32 of the sum from
// a key; at a sum of 1 it took 2^-25, and a long flat tail beside a peak was lost altogether.  Beside a bf16 cache they
// are held 2^8 times smaller, at most 1, so that O passes fp32's range only where a sum of the values does: values
// may be as large as fp32's own, and bf16 probabilities have its exponents.
//
// Operands of the matrix instructions.  E4M3 values are exact in bf16 and in fp16.  Scores: bf16 queries
// (as given) times bf16 keys, exact products.  Output: probabilities are rounded to fp16 next to fp16
// values for an E4M3 cache (2^-11 relative), to bf16 for a bf16 cache (2^-8), whose values may exceed
// fp16's range.
//
// The matrix products are taken transposed, S^T = K Q^T and O^T = V^T P^T: a lane then holds scores of
// ONE query row, reductions over keys stay mostly in the lane, and the score registers are the
// probability operand of the second product without any movement between lanes (the order of the keys
// in its K dimension is free as long as V^T is read in the same one).
//
// The rows of one sequence and key-value head are its new tokens times the group's query heads, packed:
// row r is token r / group, head r % group, so all of them share the keys read.  Two kernels:
//   stream_kernel   few rows (16 or 32): HBM-bound.  Every wavefront streams its own keys straight
//                   from memory into matrix-operand registers, no LDS in the loop, no barriers.
//   tile_kernel     many rows (128 or more): MFMA-bound.  Keys and values are converted once per
//                   workgroup on their way into LDS.
// Tiles of rows are found on the device: slot index -> sequence by a search over cu_q, since
// floor(cu_q[s] group / BM) + s is a monotone numbering that leaves every sequence enough slots.
//
// Split of the key axis: with few row tiles, the key blocks of all (head, slot) segments form one
// sequence that is cut into equal shares, one per workgroup, from the lengths as they are on the device.  A
// segment inside one share is finished there; a cut one leaves (m, l, O) per share in the workspace,
// joined by combine_kernel in a fixed order.  Equal shares are what a batch of uneven lengths needs: 64 tokens
// over caches of 512 to 32768 tokens (2.2 GB) take 406 us, 5.4 TB/s.
//
// Keys outside [0, kv_len) or on an invalid page are zeroed (V) and masked (scores); keys only some rows of
// a tile see are masked by selection.  0 * inf would still reach rows that do not see the key, so
// non-finite values of V are taken out of the product and added afterwards to the rows that do see
// them (any positive probability times inf or NaN is inf or NaN, also one too small for fp32).
#include "paged_device.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlots = 1024;       // row tiles a split launch can plan
constexpr int kStreamBlock = 128;     // keys per step of stream_kernel: 32 per wavefront
constexpr int kTileBlock = 64;        // keys per step of tile_kernel: one 16-key group per wavefront
// What cutting the key axis costs a tile_kernel launch, in key blocks: the extra prologues, the parts written and
// joined take about 20 us, a block 0.8 to 2.6 us.  Tiles are kept whole where the blocks of a workgroup, by the mean over
// the launch's slots, are no more than that above an even share: 1024 new tokens alone 45 us whole and 60 cut, over
// 32768 keys 970 whole and 760 cut.  The mean counts empty slots and says nothing of the longest tile: 4 chunks of 300
// tokens among 17 sequences (head dim 256, window 2048) stay whole with a longest tile of 34 blocks against an even
// share of 13, 114 us.
constexpr int kCutCost = 16;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLazy = 8.0f;
template <bool FP8>
constexpr float kLift = FP8 ? 7.0f : -8.0f;
// An exponent is one fused multiply-add, s c - (m c - kLift), whose constant is rounded: at the row's largest key it is off
// by half an ulp of m c, which passes 1 from |m c| = 2^24 on and would overflow or erase every probability of the row
// further up.  From this size on the scores are taken against the maximum first (below it the rounding is under 2^-12).
constexpr float kFar = 0x1p12f;
constexpr float kLn2 = 0.693147180559945f;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// What a launch adds to the call's arguments.
struct Launch {
  int32_t slots;             // row tiles, an upper bound
  int32_t rows_lo, rows_hi;  // sequences with rows in (rows_lo, rows_hi] are this launch's
  int32_t split;             // 0: one workgroup per (slot, head)
  int32_t workgroups;        // of a split launch
  int32_t min_blocks;        // smallest share
  int32_t rows_grid;         // combine_kernel: workgroups per (slot, head)
  int32_t* plan;             // written by the attention kernel for combine_kernel: [0] blocks per share, [1] all
                             // blocks of a head, [2 ..] first block of every sequence (stream) or slot (tile)
  float2* ml;                // [2 workgroups][BM]: m c - kLift, l
  float* po;                 // [2 workgroups][BM][D]: O
};

// One row tile of one sequence.
struct Tile {
  int s, c0, n, len;         // sequence, its first row of q, new tokens, cache length
  int row0, rows;            // first packed row, rows in the tile
  int pos0;                  // position of the sequence's first new token (may be negative)
  int hi_min, lo_max;        // keys in [lo_max, hi_min) are seen by every row
  int block0, blocks;        // first key block and their number (at least 1)
};

__device__ __forceinline__ int cu_at(const AttentionArgs& a, int j) { return clamp_int(a.cu_q[j], 0, a.tokens); }

// First slot of sequence s: its own number where this launch's sequences have one tile each.
template <int BM>
__device__ __forceinline__ int first_slot(const AttentionArgs& a, const Launch& l, int s) {
  return l.rows_hi <= BM ? s : (int)((uint32_t)(cu_at(a, s) * a.group) / BM) + s;
}

// Tile `i` of sequence s; false if there is none or it is another launch's.
template <int BM, int KB>
__device__ __forceinline__ bool tile_of(const AttentionArgs& a, const Launch& l, int s, int i, Tile& t) {
  t.s = s;
  t.c0 = cu_at(a, s);
  t.n = clamp_int(a.cu_q[s + 1], t.c0, a.tokens) - t.c0;
  const int all = t.n * a.group;
  if (all <= l.rows_lo || all > l.rows_hi || i < 0 || (int64_t)i * BM >= all) return false;
  t.len = clamp_int(a.kv_len[s], 0, a.table_width << a.page_shift);
  t.row0 = i * BM;
  t.rows = all - t.row0 < BM ? all - t.row0 : BM;
  t.pos0 = t.len - t.n;
  const int first = (int)fastdiv((uint32_t)t.row0, a.div_group);
  const int last = (int)fastdiv((uint32_t)(t.row0 + t.rows - 1), a.div_group);
  int hi = t.len, lo = 0;
  t.hi_min = t.len;
  t.lo_max = 0;
  if (a.causal) {
    hi = clamp_int(t.pos0 + last + 1, 0, t.len);
    t.hi_min = clamp_int(t.pos0 + first + 1, 0, t.len);
    if (a.window > 0) {
      const int64_t l0 = (int64_t)t.pos0 + first - a.window + 1, l1 = (int64_t)t.pos0 + last - a.window + 1;
      lo = l0 > 0 ? (int)l0 : 0;
      t.lo_max = l1 > 0 ? (int)l1 : 0;
    }
  }
  t.block0 = lo / KB;
  t.blocks = hi > lo ? (hi + KB - 1) / KB - t.block0 : 1;
  return true;
}

// Keys [lo, hi) that packed row r of the tile's sequence sees; none for rows past the tile.
__device__ __forceinline__ void row_range(const AttentionArgs& a, const Tile& t, int r, int& lo, int& hi) {
  lo = 0;
  hi = 0;
  if (r >= t.row0 + t.rows) return;
  hi = t.len;
  if (a.causal) {
    const int pos = t.pos0 + (int)fastdiv((uint32_t)r, a.div_group);
    hi = clamp_int(pos + 1, 0, t.len);
    if (a.window > 0) {
      const int64_t l0 = (int64_t)pos - a.window + 1;
      lo = l0 > 0 ? (int)l0 : 0;
    }
  }
}

// Page of the 16-aligned key group at `key` (16 keys never straddle a page): its number, or -1.
__device__ __forceinline__ int page_of(const AttentionArgs& a, const Tile& t, int key) {
  if (key >= t.len) return -1;
  const int p = scalar_load(a.page_table + t.s * a.table_stride + (key >> a.page_shift));
  return (uint32_t)p < (uint32_t)a.num_pages ? p : -1;
}

// ---- splitting the key axis ----------------------------------------------------------------------

// First block of every slot (pre[0 .. slots], pre[slots] = all blocks of one head), by the whole workgroup.
template <int BM, int KB>
__device__ __forceinline__ void make_plan(const AttentionArgs& a, const Launch& l, int* pre, int* wave_sum) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kPer = kMaxSlots / kThreads;
  for (int j = tid; j < kMaxSlots; j += kThreads) pre[j] = 0;
  __syncthreads();
  Tile t;
  if (a.num_seqs <= 16) {              // few sequences: threads over the tiles of each
    for (int s = 0; s < a.num_seqs; ++s) {
      const int base = first_slot<BM>(a, l, s);
      for (int i = tid; base + i < l.slots && tile_of<BM, KB>(a, l, s, i, t); i += kThreads) pre[base + i] = t.blocks;
    }
  } else {                             // many: one thread per sequence, few tiles each
    for (int s = tid; s < a.num_seqs; s += kThreads) {
      const int base = first_slot<BM>(a, l, s);
      for (int i = 0; base + i < l.slots && tile_of<BM, KB>(a, l, s, i, t); ++i) pre[base + i] = t.blocks;
    }
  }
  __syncthreads();
  int v[kPer], sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    v[j] = pre[tid * kPer + j];
    sum += v[j];
  }
  int inc = sum;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const int o = __shfl_up(inc, m, 64);
    if (lane >= m) inc += o;
  }
  if (lane == 63) wave_sum[wave] = inc;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < wave; ++w) at += wave_sum[w];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    pre[tid * kPer + j] = at;
    at += v[j];
  }
  if (tid == kThreads - 1) pre[kMaxSlots] = at;
  __syncthreads();
}

// Shares of a split launch: `per` blocks each, in order over (head, tile, block).
struct Shares {
  int64_t total;
  int per;
};

__device__ __forceinline__ Shares shares_of(const AttentionArgs& a, const Launch& l, int all) {
  const int64_t total = (int64_t)all * a.kv_heads;
  const int64_t share = (total + l.workgroups - 1) / l.workgroups;
  return Shares{total, share > l.min_blocks ? (int)share : l.min_blocks};
}

// This workgroup's share.  Workgroups are dealt to the 8 XCDs in turn; neighbouring shares (mostly the same
// head's keys) go to one XCD, and a launch with less work than workgroups still uses all XCDs.
__device__ __forceinline__ int my_share(const Shares& s) {
  const int used = (int)((s.total + s.per - 1) / s.per), each = (used + 7) >> 3;
  const int x = blockIdx.x & 7, i = blockIdx.x >> 3;
  return i < each ? x * each + i : used;
}

// A value that is the same in every lane, as the scalar it is: what follows from it (addresses, loop bounds, the
// page table's loads) then stays on the scalar unit.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The unsplit launch: one workgroup per (slot, head), late (long) tiles first.
template <int BM, int KB>
__device__ __forceinline__ bool whole_tile(const AttentionArgs& a, const Launch& l, Tile& t, int& h) {
  h = blockIdx.x % a.kv_heads;
  const int slot = l.slots - 1 - (int)(blockIdx.x / a.kv_heads);
  const int s = wave_search(a.num_seqs, [&](int j) { return first_slot<BM>(a, l, j) <= slot; });
  return s >= 0 && tile_of<BM, KB>(a, l, s, slot - first_slot<BM>(a, l, s), t);
}

// Calls work(tile, head, first block, end block, partial) for every piece of this workgroup's share; partial <
// 0: the whole tile.  Uniform over the workgroup.  Exact block counts per row tile (early tiles of a causal
// chunk see fewer keys), planned by the whole workgroup over all slots.
template <int BM, int KB, typename Work>
__device__ __forceinline__ void tile_pieces(const AttentionArgs& a, const Launch& l, int* pre, int* wave_sum, Work work) {
  Tile t;
  int64_t u = 0, end = 1;
  int all = 0, w = 0, h = 0;
  bool whole = false;
  if (l.split) {
    make_plan<BM, KB>(a, l, pre, wave_sum);
    all = uniform(pre[kMaxSlots]);
    const Shares sh = shares_of(a, l, all);
    const int units = l.slots * a.kv_heads;
    whole = (int64_t)((units + l.workgroups - 1) / l.workgroups) * all <= (int64_t)(kCutCost + sh.per) * l.slots;
    if (blockIdx.x == 0) {
      for (int j = threadIdx.x; j <= l.slots; j += kThreads) l.plan[2 + j] = pre[j];
      if (threadIdx.x == 0) {
        l.plan[0] = whole ? INT32_MAX : sh.per;
        l.plan[1] = all;
      }
    }
    if (whole) {
      u = blockIdx.x;
      end = u < units ? u + 1 : u;
    } else {
      w = my_share(sh);
      u = (int64_t)w * sh.per;
      end = u + sh.per < sh.total ? u + sh.per : sh.total;
    }
  }
  while (u < end) {
    int off = 0, take, partial = -1;
    if (whole) {
      const int unit = (int)u, slot = l.slots - 1 - unit / a.kv_heads;
      h = unit % a.kv_heads;
      u = end;
      const int s = wave_search(a.num_seqs, [&](int j) { return first_slot<BM>(a, l, j) <= slot; });
      if (s < 0 || !tile_of<BM, KB>(a, l, s, slot - first_slot<BM>(a, l, s), t)) continue;
      take = t.blocks;
    } else if (l.split) {
      h = (int)(u / all);
      const int rem = (int)(u - (int64_t)h * all);
      int lo = 0, hi = l.slots;                   // pre[lo] <= rem < pre[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (uniform(pre[mid]) <= rem) lo = mid; else hi = mid;
      }
      const int first = uniform(pre[lo]), count = uniform(pre[lo + 1]) - first;
      off = rem - first;
      take = end - u < count - off ? (int)(end - u) : count - off;
      u += take;
      const int s = wave_search(a.num_seqs, [&](int j) { return first_slot<BM>(a, l, j) <= lo; });
      if (s < 0 || !tile_of<BM, KB>(a, l, s, lo - first_slot<BM>(a, l, s), t)) continue;
      if (take != count) partial = 2 * w + (off > 0 ? 0 : 1);
    } else {
      u = end;
      if (!whole_tile<BM, KB>(a, l, t, h)) return;
      take = t.blocks;
    }
    work(t, h, off, off + take, partial);
  }
}

// Row tiles of sequence s in this launch, and the key blocks given to each of them: those of the whole
// sequence (its new tokens are few here, so its tiles see nearly the same keys).
template <int BM, int KB>
__device__ __forceinline__ int sequence_tiles(const AttentionArgs& a, const Launch& l, int s, int& block0, int& blocks) {
  const int c0 = cu_at(a, s), n = clamp_int(a.cu_q[s + 1], c0, a.tokens) - c0, rows = n * a.group;
  const int len = clamp_int(a.kv_len[s], 0, a.table_width << a.page_shift);
  const int64_t lo = a.window > 0 ? (int64_t)len - n - a.window + 1 : 0;
  block0 = lo > 0 ? (int)lo / KB : 0;
  const int nb = (len + KB - 1) / KB - block0;
  blocks = nb > 1 ? nb : 1;
  return rows > l.rows_lo && rows <= l.rows_hi ? (rows + BM - 1) / BM : 0;
}

// As tile_pieces, planned by every wavefront for itself over the sequences, 64 at a time: one round of
// loads and a scan, no barrier.  All wavefronts write the same values to `pre`, so each may read it back at
// once.
template <int BM, int KB, typename Work>
__device__ __forceinline__ void stream_pieces(const AttentionArgs& a, const Launch& l, int* pre, Work work) {
  const int lane = threadIdx.x & 63;
  Tile t;
  int64_t u = 0, end = 1;
  int all = 0, w = 0, h = 0;
  if (l.split) {
    for (int s0 = 0; s0 < a.num_seqs; s0 += 64) {
      const int s = s0 + lane;
      int units = 0, block0, blocks;
      if (s < a.num_seqs) units = sequence_tiles<BM, KB>(a, l, s, block0, blocks) * blocks;
      int inc = units;
#pragma unroll
      for (int m = 1; m < 64; m *= 2) {
        const int o = __shfl_up(inc, m, 64);
        if (lane >= m) inc += o;
      }
      if (s < a.num_seqs) pre[s] = all + inc - units;
      all += __builtin_amdgcn_readlane(inc, 63);
    }
    if (lane == 0) pre[a.num_seqs] = all;
    const Shares sh = shares_of(a, l, all);
    if (blockIdx.x == 0 && threadIdx.x < 64) {
      for (int j = lane; j <= a.num_seqs; j += 64) l.plan[2 + j] = pre[j];
      if (lane == 0) {
        l.plan[0] = sh.per;
        l.plan[1] = all;
      }
    }
    w = my_share(sh);
    u = (int64_t)w * sh.per;
    end = u + sh.per < sh.total ? u + sh.per : sh.total;
  }
  while (u < end) {
    int off = 0, take, partial = -1;
    if (l.split) {
      h = (int)(u / all);
      const int rem = (int)(u - (int64_t)h * all);
      const int s = wave_search(a.num_seqs, [&](int j) { return pre[j] <= rem; });
      int block0, blocks;
      const int tiles = sequence_tiles<BM, KB>(a, l, s, block0, blocks);
      const int at = rem - uniform(pre[s]), i = at / blocks;
      off = at - i * blocks;
      take = end - u < blocks - off ? (int)(end - u) : blocks - off;
      u += take;
      if (i >= tiles || !tile_of<BM, KB>(a, l, s, i, t)) continue;
      t.block0 = block0;
      t.blocks = blocks;
      if (take != blocks) partial = 2 * w + (off > 0 ? 0 : 1);
    } else {
      u = end;
      if (!whole_tile<BM, KB>(a, l, t, h)) return;
      take = t.blocks;
    }
    work(t, h, off, off + take, partial);
  }
}

// ---- operand helpers -------------------------------------------------------------------------------

// Four E4M3 bytes of a dword as fp16 / bf16 pairs (exact; 0x7F and 0xFF become NaN).
__device__ __forceinline__ uint32_t fp8_bf16(uint32_t w, bool high) {
  return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
__device__ __forceinline__ uint32_t fp8_f16(uint32_t w, bool high) {
  return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){lo, hi}, half2_t));
}
template <bool FP8>
__device__ __forceinline__ uint32_t p_pair(float lo, float hi) {
  return FP8 ? f16_pair(lo, hi) : bf16_pair(lo, hi);
}

// Element t of 8 keys' dwords a[j] (E4M3: 4 elements a dword, bf16: 2), as an 8-long operand in key order.
// All elements of the dwords at once: out[t] for t = 0 .. 3 (or 0, 1).
__device__ __forceinline__ void transpose_fp8(const uint32_t (&a)[8], u32x4_t (&out)[4]) {
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t *x = a + 4 * half;
    const uint32_t p = __builtin_amdgcn_perm(x[1], x[0], 0x05010400u), q = __builtin_amdgcn_perm(x[1], x[0], 0x07030602u);
    const uint32_t r = __builtin_amdgcn_perm(x[3], x[2], 0x05010400u), s = __builtin_amdgcn_perm(x[3], x[2], 0x07030602u);
    uint32_t* o = half ? hi : lo;
    o[0] = __builtin_amdgcn_perm(r, p, 0x05040100u);
    o[1] = __builtin_amdgcn_perm(r, p, 0x07060302u);
    o[2] = __builtin_amdgcn_perm(s, q, 0x05040100u);
    o[3] = __builtin_amdgcn_perm(s, q, 0x07060302u);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
    out[t] = u32x4_t{fp8_f16(lo[t], false), fp8_f16(lo[t], true), fp8_f16(hi[t], false), fp8_f16(hi[t], true)};
}
__device__ __forceinline__ void transpose_bf16(const uint32_t (&a)[8], u32x4_t (&out)[2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[0][i] = __builtin_amdgcn_perm(a[2 * i + 1], a[2 * i], 0x05040100u);
    out[1][i] = __builtin_amdgcn_perm(a[2 * i + 1], a[2 * i], 0x07060302u);
  }
}

// Bits that are set in every non-finite element of a dword of the cache (E4M3 NaN bytes, bf16 inf or NaN).
template <bool FP8>
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
  return FP8 ? ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u;
}

// The dword without its non-finite elements.
template <bool FP8>
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  const uint32_t bits = non_finite<FP8>(w);
  return FP8 ? w & ~((bits >> 7) * 0xFFu) : w & ~((bits >> 15) * 0xFFFFu);
}

// Which of a dword's elements are +inf or NaN (`up`), and -inf or NaN (`down`), one bit each; E4M3 has NaN only.
template <bool FP8>
__device__ __forceinline__ void non_finite_signs(uint32_t w, uint32_t& up, uint32_t& down) {
  up = down = 0;
  const uint32_t nf = non_finite<FP8>(w);
#pragma unroll
  for (int e = 0; e < (FP8 ? 4 : 2); ++e) {
    const bool is = (nf >> (FP8 ? 8 * e + 7 : 16 * e + 15)) & 1;
    const bool nan = FP8 || ((w >> (16 * e)) & 0x7Fu) != 0;
    const bool neg = !FP8 && ((w >> (16 * e + 15)) & 1);
    up |= (is && (nan || !neg) ? 1u : 0u) << e;
    down |= (is && (nan || neg) ? 1u : 0u) << e;
  }
}

__device__ __forceinline__ f32x4_t mfma16_bf16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
template <bool FP8>
__device__ __forceinline__ f32x4_t mfma16_pv(u32x4_t a, u32x4_t b, f32x4_t c) {
  if (FP8)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  return mfma16_bf16(a, b, c);
}
__device__ __forceinline__ f32x16_t mfma32_bf16(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
template <bool FP8>
__device__ __forceinline__ f32x16_t mfma32_pv(u32x4_t a, u32x4_t b, f32x16_t c) {
  if (FP8)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  return mfma32_bf16(a, b, c);
}

// What the non-finite values of V that a row sees add to an output.
__device__ __forceinline__ float non_finite_part(uint32_t up, uint32_t down) {
  return (up ? __builtin_inff() : 0.0f) + (down ? -__builtin_inff() : 0.0f);
}

// A part's O times its weight, at most 1.  An infinite or NaN O (from such values, under positive probabilities) stays
// what it is also where the weight underflows to 0: the answer does not depend on how the keys were divided.  Joins
// multiply plainly (KEEP false) and are done again with KEEP where that gives a NaN, which is rare (selecting always: one
// token over 4096 keys 12.8 us a captured call, so 12.1).
template <bool KEEP>
__device__ __forceinline__ float weighted(float o, float w) {
  const float x = o * w;
  return KEEP && x != x ? o : x;
}
template <bool KEEP>
struct Keep {
  static constexpr bool value = KEEP;
};

// O / l v_scale (f is 1 / l; v_scale / l could underflow where the product does not).  A row whose sum is 0 has zeros,
// selected and not multiplied: its O may be infinite or NaN, from values at keys whose scores are all -inf.
__device__ __forceinline__ float normalised(float o, float l, float f, float vs) { return l == 0.0f ? 0.0f : o * f * vs; }

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (W == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  }
}

// Maximum and sum of x over lanes 32 apart (and, for the 16-row kernel, 16 apart): the two swapped halves.
__device__ __forceinline__ float max_across_32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_across_16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// What a row's exponents are taken against, m c - kLift, from its running maximum; 0 while that is the lowest value: a
// row that has seen no key (its scores are -inf, their exponentials 0 beside any finite value), or one whose
// scores are all so small beside 1 / c that the maximum has not moved (c below 2.4e-38).
template <bool FP8>
__device__ __forceinline__ float exponent_base(float m, float c) {
  return m == kLowest ? 0.0f : __builtin_fmaf(m, c, -kLift<FP8>);
}
// The same for joining parts, where a row without a sum must not weigh: the lowest value.  Kept finite, as the
// difference of two parts' has to be.
template <bool FP8>
__device__ __forceinline__ float scaled_max(float m, float c, float sum) {
  return sum == 0.0f ? kLowest : __builtin_amdgcn_fmed3f(exponent_base<FP8>(m, c), kLowest, -kLowest);
}
// The factor that brings what was summed against maximum m to maximum mx.
template <bool FP8>
__device__ __forceinline__ float rescale(float m, float mx, float c) {
  return exp2_fast(m == kLowest ? __builtin_fminf(-exponent_base<FP8>(mx, c), 0.0f) : (m - mx) * c);
}
// Whether any row of the wavefront has to have its scores taken against the maximum first.  Looked at in every block:
// with a flag kept from the maximum's last change, or in one branch with the change, the compiler lays the loop out
// twice and spills (8192 new tokens, head dim 128: 1030 and 985 us, so 753).
__device__ __forceinline__ bool far_scores(float base) {
  return __builtin_amdgcn_ballot_w64(__builtin_fabsf(base) > kFar) != 0;
}

// ---- few rows ----------------------------------------------------------------------------------------

// Wavefronts per SIMD of the instances, by an estimate of their registers (queries, O, one block of K and of V).  It is a
// little low for two: <64, E4M3, 2 row blocks> at 128 registers and <256, bf16, 2> at 512 keep 52 and 40 bytes a lane in
// scratch.
constexpr int stream_waves(int d, bool fp8, int rb) {
  const int regs = rb * (d / 8 + d / 4) + d / 4 * (fp8 ? 1 : 2) + 64;
  return regs <= 128 ? 4 : (regs <= 168 ? 3 : (regs <= 256 ? 2 : 1));
}

// HBM-bound: 2.2 GB of E4M3 cache in 397 us (379 to 401; 5.5 TB/s, where a plain streaming read of as much reaches 6.3),
// 143 MB of bf16 cache in 31 us (4.7 TB/s).  Registers, not LDS, hold the operands because no wavefront shares keys
// with another; one block of K and one of V in flight per wavefront at three wavefronts per SIMD cover the latency (two
// blocks at two wavefronts: 493 us).  Page numbers come through scalar loads: as vector loads they waited for the keys
// and values in flight (480 us).
// RB blocks of 16 rows; lane n = lane % 16 is the row, quarter = lane / 16.
//   scores   S^T[g] (16 keys x 16 rows): lane holds keys g*16 + quarter*4 + i of its row
//   K        A operand, lane = key, quarter = slice of the channels: 16 B loads, two matrix steps each
//            for E4M3 (channels c*64 + quarter*16 + half*8 + j), one for bf16 (c*32 + quarter*8 + j); the
//            queries are loaded in the same channel order
//   V        lane % 16 = slice of D/16 channels, quarter = 8 keys (quarter*4 + j of both groups); bytes
//            transposed in registers to A operands of 16 channels x 32 keys: O^T tile t holds
//            channels (quarter*4 + i) * D/16 + t
template <int D, bool FP8, int RB>
__global__ __launch_bounds__(kThreads, stream_waves(D, FP8, RB)) void stream_kernel(AttentionArgs a, Launch l) {
  constexpr int E = FP8 ? 1 : 2;            // bytes per element
  constexpr int BM = 16 * RB;
  constexpr int KC = D * E / 64;            // 16-byte key loads per lane and group
  constexpr int ST = D / 32;                // matrix steps of a score
  constexpr int NT = D / 16;                // output tiles, and channels per lane slice
  constexpr int VW = NT * E / 4;            // dwords of V per lane and key
  constexpr int PT = D + 4;                 // LDS pitch of the merge
  constexpr int MW = (D / 4 + 31) / 32;     // dwords of marks: a bit per output of a lane
  __shared__ __align__(16) float merge[4][16][PT];
  uint32_t* const marks = reinterpret_cast<uint32_t*>(merge);      // in the loop, before the merge
  static_assert(RB * 2 * MW * kThreads <= 4 * 16 * PT, "marks fit the merge buffer");
  __shared__ float2 merge_ml[4][16];
  __shared__ int pre[kMaxSlots + 1];

  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  stream_pieces<BM, kStreamBlock>(a, l, pre, [&](const Tile& t, int h, int b0, int b1, int partial) {
    const float c = a.scale_log2 * (FP8 ? a.k_scale[h * a.scale_stride] : 1.0f);
    u32x4_t q[RB][ST];
    int lo[RB], hi[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = t.row0 + rb * 16 + n;
      row_range(a, t, r, lo[rb], hi[rb]);
      const bool live = rb * 16 + n < t.rows;
      const int tok = (int)fastdiv((uint32_t)r, a.div_group), g = r - tok * a.group;
      const uint16_t* x = a.q + (live ? (t.c0 + tok) * a.q_tok + (h * a.group + g) * a.q_head : 0);
#pragma unroll
      for (int st = 0; st < ST; ++st) {
        const int d = FP8 ? (st >> 1) * 64 + quarter * 16 + (st & 1) * 8 : st * 32 + quarter * 8;
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(x + d);
        q[rb][st] = live ? w : u32x4_t{0, 0, 0, 0};
      }
    }
    f32x4_t o[RB][NT];
    float m[RB], sum[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      m[rb] = kLowest;
      sum[rb] = 0.0f;
#pragma unroll
      for (int i = 0; i < NT; ++i) o[rb][i] = f32x4_t{0, 0, 0, 0};
    }

    const int64_t head_at = ((int64_t)h << a.page_shift) * (D * E);
    const int mask = (1 << a.page_shift) - 1;
    auto key_at = [&](int b) { return (t.block0 + b) * kStreamBlock + wave * 32; };
    auto pages = [&](int b, int (&p)[2]) {
      p[0] = b < b1 ? page_of(a, t, key_at(b)) : -1;
      p[1] = b < b1 ? page_of(a, t, key_at(b) + 16) : -1;
    };
    uint4 kr[2][KC];
    uint32_t vr[8][VW];
    auto load_k = [&](int b, const int (&p)[2]) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int in = (key_at(b) + g * 16) & mask, page = p[g] >= 0 ? p[g] : 0;
        const uint8_t* kp = a.k + page * a.k_page + head_at + in * (D * E);
#pragma unroll
        for (int i = 0; i < KC; ++i) kr[g][i] = *reinterpret_cast<const uint4*>(kp + n * (D * E) + i * 64 + quarter * 16);
      }
    };
    auto load_v = [&](int b, const int (&p)[2]) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int in = (key_at(b) + g * 16) & mask, page = p[g] >= 0 ? p[g] : 0;
        const uint8_t* vp = a.v + page * a.v_page + head_at + in * (D * E);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_words<VW>(vp + (quarter * 4 + j) * (D * E) + n * (NT * E), vr[g * 4 + j]);
      }
    };

    // One block at a time: V of this block and K of the next are in flight while the other is used.
    bool marked = false;
    __syncthreads();                          // the last piece's merge has been read
    int p[2], pn[2], pv[2];
    pages(b0, p);
    load_k(b0, p);
    pages(b0 + 1, pn);
    for (int b = b0; b < b1; ++b) {
      const int key0 = key_at(b), valid = (p[0] >= 0 ? 1 : 0) | (p[1] >= 0 ? 2 : 0);
      load_v(b, p);
      f32x4_t s[RB][2];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) s[rb][0] = s[rb][1] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          u32x4_t ka;
          if (FP8) {
            const uint4 w = kr[g][st >> 1];
            const uint32_t x = st & 1 ? w.z : w.x, y = st & 1 ? w.w : w.y;
            ka = u32x4_t{fp8_bf16(x, false), fp8_bf16(x, true), fp8_bf16(y, false), fp8_bf16(y, true)};
          } else {
            const uint4 w = kr[g][st];
            ka = u32x4_t{w.x, w.y, w.z, w.w};
          }
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) s[rb][g] = mfma16_bf16(ka, q[rb][st], s[rb][g]);
        }
      if (b + 1 < b1) load_k(b + 1, pn);
      pv[0] = p[0];
      pv[1] = p[1];
      p[0] = pn[0];
      p[1] = pn[1];
      pages(b + 2, pn);

      const bool partial_keys = valid != 3 || key0 + 32 > t.hi_min || key0 < t.lo_max;
      u32x4_t pr[RB] = {};
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        if (partial_keys) {
          asm volatile("");        // a branch, not selects paid by every block
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = key0 + g * 16 + quarter * 4 + i;
              const bool seen = ((valid >> g) & 1) && key >= lo[rb] && key < hi[rb];
              s[rb][g][i] = seen ? s[rb][g][i] : -__builtin_inff();
            }
        }
        float mx = m[rb];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = __builtin_fmaxf(mx, s[rb][g][i]);
        mx = max_across_32(max_across_16(mx));
        if (__builtin_amdgcn_ballot_w64((mx - m[rb]) * c > kLazy) != 0) {
          const float f0 = rescale<FP8>(m[rb], mx, c);
          m[rb] = mx;
          sum[rb] *= f0;
#pragma unroll
          for (int i = 0; i < NT; ++i) o[rb][i] *= f0;
        }
        float mc = exponent_base<FP8>(m[rb], c);
        if (far_scores(mc)) {
          asm volatile("");        // a branch, as above
          const float from = m[rb] == kLowest ? 0.0f : m[rb];
#pragma unroll
          for (int j = 0; j < 8; ++j) s[rb][j >> 2][j & 3] -= from;
          mc = -kLift<FP8>;
        }
        float p8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p8[j] = exp2_fast(__builtin_fmaf(s[rb][j >> 2][j & 3], c, -mc));
          sum[rb] += p8[j];
          if (j & 1) pr[rb][j >> 1] = p_pair<FP8>(p8[j - 1], p8[j]);
        }
      }

      if (valid != 3 || key0 + 32 > t.len) {             // keys that do not exist: zero their values
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool there = ((valid >> (j >> 2)) & 1) && key0 + (j >> 2) * 16 + quarter * 4 + (j & 3) < t.len;
#pragma unroll
          for (int i = 0; i < VW; ++i) vr[j][i] = there ? vr[j][i] : 0u;
        }
      }
      uint32_t bad = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < VW; ++i) bad |= non_finite<FP8>(vr[j][i]);
      const bool any_bad = __builtin_amdgcn_ballot_w64(bad != 0) != 0;
      constexpr int PER = FP8 ? 4 : 2;
      if (any_bad) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < VW; ++i) vr[j][i] = finite_part<FP8>(vr[j][i]);
      }
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = vr[j][i];
        u32x4_t va[PER];
        if constexpr (FP8) transpose_fp8(w, va); else transpose_bf16(w, va);
#pragma unroll
        for (int x = 0; x < PER; ++x)
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) o[rb][i * PER + x] = mfma16_pv<FP8>(va[x], pr[rb], o[rb][i * PER + x]);
      }
      if (any_bad) {
        // Rare: mark this lane's outputs that see a non-finite value, by reading the block's values again.
        if (!marked)
          for (int i = 0; i < RB * 2 * MW; ++i) marks[i * kThreads + tid] = 0;
        marked = true;
#pragma unroll 1
        for (int kk = 0; kk < 32; ++kk) {
          const int key = key0 + kk, page = kk < 16 ? pv[0] : pv[1];
          if (key >= t.len || page < 0) continue;
          const uint8_t* vp = a.v + page * a.v_page + head_at + (key & mask) * (D * E) + quarter * (4 * NT * E);
          uint32_t seen = 0;
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) seen |= (key >= lo[rb] && key < hi[rb] ? 1u : 0u) << rb;
#pragma unroll 1
          for (int i = 0; i < NT * E; ++i) {           // the dwords of 4 slices of NT channels
            uint32_t up, down;
            non_finite_signs<FP8>(*reinterpret_cast<const uint32_t*>(vp + 4 * i), up, down);
            const int bit = i * PER;
            for (int rb = 0; rb < RB; ++rb) {
              if (!((seen >> rb) & 1)) continue;
              marks[((rb * 2) * MW + (bit >> 5)) * kThreads + tid] |= up << (bit & 31);
              marks[((rb * 2 + 1) * MW + (bit >> 5)) * kThreads + tid] |= down << (bit & 31);
            }
          }
        }
      }
    }
    if (marked) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int bit = x * NT + i;
            o[rb][i][x] += non_finite_part((marks[((rb * 2) * MW + (bit >> 5)) * kThreads + tid] >> (bit & 31)) & 1,
                                           (marks[((rb * 2 + 1) * MW + (bit >> 5)) * kThreads + tid] >> (bit & 31)) & 1);
          }
    }

    // the four wavefronts' parts, 16 rows at a time
    const float vs = FP8 ? a.v_scale[h * a.scale_stride] : 1.0f;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      float l0 = sum[rb];
      l0 += __shfl_xor(l0, 16, 64);
      l0 += __shfl_xor(l0, 32, 64);
      __syncthreads();
      if (quarter == 0) merge_ml[wave][n] = make_float2(scaled_max<FP8>(m[rb], c, l0), l0);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int i = 0; i < NT; i += 4)
          *reinterpret_cast<f32x4_t*>(&merge[wave][n][(quarter * 4 + x) * NT + i]) =
              f32x4_t{o[rb][i][x], o[rb][i + 1][x], o[rb][i + 2][x], o[rb][i + 3][x]};
      __syncthreads();
      const int row = tid >> 4, d = (tid & 15) * NT;
      if (rb * 16 + row < t.rows) {
        float mm = kLowest, ll = 0.0f, w[4], e[NT];
#pragma unroll
        for (int v = 0; v < 4; ++v) mm = __builtin_fmaxf(mm, merge_ml[v][row].x);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          w[v] = exp2_fast(merge_ml[v][row].x - mm);
          ll += merge_ml[v][row].y * w[v];
        }
        auto join = [&](auto keep) {
          float all = 0.0f;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            e[i] = 0.0f;
#pragma unroll
            for (int v = 0; v < 4; ++v) e[i] += weighted<decltype(keep)::value>(merge[v][row][d + i], w[v]);
            all += e[i];
          }
          return all != all;
        };
        if (join(Keep<false>{})) join(Keep<true>{});
        if (partial >= 0) {
          const int64_t at = (int64_t)partial * BM + rb * 16 + row;
          if (d == 0) l.ml[at] = make_float2(mm, ll);
#pragma unroll
          for (int i = 0; i < NT; i += 4)
            *reinterpret_cast<float4*>(l.po + at * D + d + i) = make_float4(e[i], e[i + 1], e[i + 2], e[i + 3]);
        } else {
          const int r = t.row0 + rb * 16 + row;
          const int tok = (int)fastdiv((uint32_t)r, a.div_group), head = h * a.group + r - tok * a.group;
          const float f = 1.0f / ll;
          uint16_t* y = a.out + (t.c0 + tok) * a.o_tok + head * a.o_head + d;
#pragma unroll
          for (int i = 0; i < NT; i += 4)
            *reinterpret_cast<uint2*>(y + i) =
                make_uint2(bf16_pair(normalised(e[i], ll, f, vs), normalised(e[i + 1], ll, f, vs)),
                           bf16_pair(normalised(e[i + 2], ll, f, vs), normalised(e[i + 3], ll, f, vs)));
          if (a.lse && d == 0) a.lse[(int64_t)(t.c0 + tok) * a.q_heads + head] = (mm + __builtin_log2f(ll)) * kLn2;
        }
      }
    }
  });
}

// Ends a step of a hand-ordered instruction sequence.  Left to itself the compiler reads each LDS operand right
// before its use, waits out the latency for every matrix instruction, and puts all exponentials in front of
// all products; with a boundary after every matrix instruction the reads run four ahead and the vector
// instructions between two products execute while the matrix pipe is busy.
__device__ __forceinline__ void step() { __builtin_amdgcn_sched_barrier(0); }

// ---- many rows ---------------------------------------------------------------------------------------

// MFMA-bound in principle; in fact neither pipe is full: 8192 new tokens of 40 heads of 128 in 745 to 800 us over
// several runs (860 to 920 TFLOP/s; an 8192^3 bf16 library product reaches 1410 here), the matrix pipe busy 42 % of
// the time, vector instructions about as much.  A bf16 cache 805 to 830 us (its instance keeps 52 bytes a lane in
// scratch).  Per wavefront and block 32 matrix instructions (32 cycles each) stand beside about 250 vector instructions,
// of which softmax's 32 scores a lane take 130 and the staging of the next block 75.  A single wavefront issues a
// vector instruction every 8 cycles, two every 4 (measured), so two wavefronts per SIMD are needed and everything that
// can goes between matrix instructions: staging into the score product, exponentials into the second (837 -> 727 us for
// both).  64 rows a wavefront (half the LDS reads, one wavefront per SIMD) is slower: 814 us; so is output through LDS
// in whole rows (no gain, more registers).  Head dim 256 has registers for one wavefront per SIMD only: 1710 us, 804
// TFLOP/s.
// Four wavefronts of 32 rows each; lane % 32 is the row, half = lane / 32.
//   scores   S^T (32 keys x 32 rows): register i of a lane is key 8*(i/4) + 4*half + i%4
//   LDS      K as bf16 [key][D] and V^T as fp16 or bf16 [D][64 keys], both double-buffered, in 16-byte
//            chunks permuted within a row so that neighbouring rows fall on different banks.  The
//            keys of a V^T row are stored in the order the score registers hold them: chunk
//            2*(key/16) + half holds keys 4*half + {0..3} and 8 + 4*half + {0..3} of its 16.
template <int I>
struct Buffer {
  static constexpr int value = I;
};

template <int D, bool FP8>
__global__ __launch_bounds__(kThreads, D <= 128 ? 2 : 1) void tile_kernel(AttentionArgs a, Launch l) {
  constexpr int E = FP8 ? 1 : 2;
  constexpr int BM = 128, KB = kTileBlock;
  // With one wavefront per SIMD half of its 512 registers are accumulation registers, which only matrix
  // instructions and loads address: the output and the queries are kept there.
  constexpr bool kAcc = D > 128;
  constexpr int ST = D / 16;                // matrix steps of a score
  constexpr int DB = D / 32;                // output tiles
  constexpr int CH = D * E / 16;            // 16-byte chunks of a cached key
  constexpr int NG = KB / 16;               // 16-key groups of a block, each brought in by one wavefront
  constexpr int KL = 16 * CH / 64;          // key loads per lane
  constexpr int VQ = D / 4;                 // channel quads
  constexpr int VI = VQ > 32 ? VQ / 32 : 1; // value items per lane: 8 keys x 4 channels
  __shared__ __align__(16) uint16_t ks[2][KB * D];
  __shared__ __align__(16) uint16_t vt[2][D * KB];
  __shared__ int pre[kMaxSlots + 1];
  __shared__ int wave_sum[4];
  __shared__ int bad_block[2];              // block whose values hold something non-finite
  __shared__ int no_page[2][NG];            // per 16 keys of a block
  constexpr int MW = D / 64;                // dwords of marks: a bit per output of a lane
  __shared__ uint32_t marks[2 * MW][kThreads];

  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  auto k_chunk = [](int key, int ch) {       // LDS offset (elements) of 8 channels of a key
    constexpr int N = D / 8;
    const int sw = N >= 16 ? key & 15 : (key >> 1) & 7;
    return key * D + ((ch ^ sw) & (N - 1)) * 8;
  };
  auto v_chunk = [](int d, int ch) {         // LDS offset of 8 keys of a channel
    const int sw = ((d >> 1) & 7) ^ ((d >> 4) & 1);
    return d * KB + ((ch ^ sw) & (KB / 8 - 1)) * 8;
  };

  const int v_quad = lane % VQ;
  // which 8 of its 16-key group a value item holds
  auto v_grp = [&](int i) { return VI > 1 ? i : (lane / VQ) & 1; };

  tile_pieces<BM, KB>(a, l, pre, wave_sum, [&](const Tile& t, int h, int b0, int b1, int partial) {
    const float c = a.scale_log2 * (FP8 ? a.k_scale[h * a.scale_stride] : 1.0f);
    const int wrow = wave * 32;              // the wavefront's first row in the tile
    const bool busy = wrow < t.rows;
    u32x4_t q[ST];
    int lo, hi;
    {
      const int r = t.row0 + wrow + n;
      row_range(a, t, r, lo, hi);
      const bool live = wrow + n < t.rows;
      const int tok = (int)fastdiv((uint32_t)r, a.div_group), g = r - tok * a.group;
      const uint16_t* x = a.q + (live ? (t.c0 + tok) * a.q_tok + (h * a.group + g) * a.q_head : 0);
#pragma unroll
      for (int st = 0; st < ST; ++st) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(x + st * 16 + half * 8);
        q[st] = live ? w : u32x4_t{0, 0, 0, 0};
      }
    }
    // keys every row of the wavefront sees, and keys any of them sees
    int w_first = 0, w_last = 0;
    if (busy) {
      const int rl = wrow + 32 < t.rows ? wrow + 31 : t.rows - 1;
      w_first = (int)fastdiv((uint32_t)(t.row0 + wrow), a.div_group);
      w_last = (int)fastdiv((uint32_t)(t.row0 + rl), a.div_group);
    }
    int hi_min = t.len, hi_max = t.len, lo_min = 0, lo_max = 0;
    if (a.causal) {
      hi_min = clamp_int(t.pos0 + w_first + 1, 0, t.len);
      hi_max = clamp_int(t.pos0 + w_last + 1, 0, t.len);
      if (a.window > 0) {
        const int64_t l0 = (int64_t)t.pos0 + w_first - a.window + 1, l1 = (int64_t)t.pos0 + w_last - a.window + 1;
        lo_min = l0 > 0 ? (int)l0 : 0;
        lo_max = l1 > 0 ? (int)l1 : 0;
      }
    }

    if constexpr (kAcc) {
#pragma unroll
      for (int st = 0; st < ST; ++st) asm volatile("" : "+a"(q[st]));
    }
    f32x16_t o[DB];
    float m = kLowest, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[i][x] = 0.0f;

    const int64_t head_at = ((int64_t)h << a.page_shift) * (D * E);
    const int mask = (1 << a.page_shift) - 1;
    u32x4_t kr[KL];
    uint32_t vr[VI][8][E];                   // 4 channels of 8 keys
    // Wavefront w brings in the 16-key group w of a block, which lies in one page: rows 16 w .. of K, and of V the two
    // sets of 8 keys that a 16-byte chunk of a V^T row holds.
    const int my_group = wave;
    auto my_page = [&](int b) { return b < b1 ? page_of(a, t, (t.block0 + b) * KB + my_group * 16) : -1; };
    auto fetch = [&](int b, int p) {
      const int in = ((t.block0 + b) * KB + my_group * 16) & mask;
      const uint8_t* kp = a.k + (p >= 0 ? p : 0) * a.k_page + head_at + in * (D * E);
      const uint8_t* vp = a.v + (p >= 0 ? p : 0) * a.v_page + head_at + in * (D * E);
#pragma unroll
      for (int i = 0; i < KL; ++i) kr[i] = *reinterpret_cast<const u32x4_t*>(kp + (i * 64 + lane) * 16);
#pragma unroll
      for (int i = 0; i < VI; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          load_words<E>(vp + ((j & 3) + (j >> 2) * 8 + v_grp(i) * 4) * (D * E) + v_quad * (4 * E), vr[i][j]);
    };
    // From registers to LDS, in NU small units that the score product takes in between its matrix instructions:
    // keys (one converted 16-byte chunk each), values (a few byte moves, or one channel's 8 keys), and the search
    // for non-finite values.  A tail or a missing page is zeroed first, non-finite values are taken out and
    // the values written again after: both are rare.
    constexpr int NK = FP8 ? 2 * KL : KL, PER = FP8 ? 4 : 2, NV = VI * E * (FP8 ? 8 : 2), NB = VI * E * 2;
    constexpr int NU = NK + NV + NB;
    uint32_t tv[VI * E][8];
    uint32_t bad = 0;
    auto stage_begin = [&](int b, int p, int buf) {
      const int key0 = (t.block0 + b) * KB + my_group * 16;
      if (lane == 0) no_page[buf][my_group] = p < 0;
      bad = 0;
      if (p < 0 || key0 + 16 > t.len) {      // keys that do not exist
        asm volatile("");
#pragma unroll
        for (int i = 0; i < VI; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int x = 0; x < E; ++x)
              vr[i][j][x] = p >= 0 && key0 + (j & 3) + (j >> 2) * 8 + v_grp(i) * 4 < t.len ? vr[i][j][x] : 0u;
      }
    };
    auto stage_unit = [&](int u, int buf) {
      if (u < NK) {
        const int i = FP8 ? u / 2 : u, at = i * 64 + lane, key = wave * 16 + at / CH, ch = at % CH;
        if (FP8) {
          const uint32_t lo = kr[i][(u & 1) * 2], hi = kr[i][(u & 1) * 2 + 1];
          *reinterpret_cast<u32x4_t*>(&ks[buf][k_chunk(key, 2 * ch + (u & 1))]) =
              u32x4_t{fp8_bf16(lo, false), fp8_bf16(lo, true), fp8_bf16(hi, false), fp8_bf16(hi, true)};
        } else {
          *reinterpret_cast<u32x4_t*>(&ks[buf][k_chunk(key, ch)]) = kr[i];
        }
      } else if (u < NK + NB) {
        const int v = (u - NK) / 2, h4 = (u - NK) & 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) bad |= non_finite<FP8>(vr[v / E][h4 * 4 + j][v % E]);
      } else {
        const int v = (u - NK - NB) / (FP8 ? 8 : 2), s = (u - NK - NB) % (FP8 ? 8 : 2);
        auto w = [&](int j) { return vr[v / E][j][v % E]; };
        auto put = [&](int y, u32x4_t x) {
          *reinterpret_cast<u32x4_t*>(&vt[buf][v_chunk(v_quad * 4 + (v % E) * PER + y, my_group * 2 + v_grp(v / E))]) = x;
        };
        if (FP8) {
          uint32_t(&z)[8] = tv[v];
          const int o = (s >> 1) * 4;         // keys 0..3 then 4..7
          if (s < 4 && !(s & 1)) {
            z[o] = __builtin_amdgcn_perm(w(o + 1), w(o), 0x05010400u);
            z[o + 1] = __builtin_amdgcn_perm(w(o + 1), w(o), 0x07030602u);
            z[o + 2] = __builtin_amdgcn_perm(w(o + 3), w(o + 2), 0x05010400u);
            z[o + 3] = __builtin_amdgcn_perm(w(o + 3), w(o + 2), 0x07030602u);
          } else if (s < 4) {
            const uint32_t c0 = __builtin_amdgcn_perm(z[o + 2], z[o], 0x05040100u);
            const uint32_t c1 = __builtin_amdgcn_perm(z[o + 2], z[o], 0x07060302u);
            const uint32_t c2 = __builtin_amdgcn_perm(z[o + 3], z[o + 1], 0x05040100u);
            const uint32_t c3 = __builtin_amdgcn_perm(z[o + 3], z[o + 1], 0x07060302u);
            z[o] = c0; z[o + 1] = c1; z[o + 2] = c2; z[o + 3] = c3;
          } else {
            const int y = s - 4;
            put(y, u32x4_t{fp8_f16(z[y], false), fp8_f16(z[y], true), fp8_f16(z[4 + y], false), fp8_f16(z[4 + y], true)});
          }
        } else {
          const uint32_t sel = s ? 0x07060302u : 0x05040100u;
          put(s, u32x4_t{__builtin_amdgcn_perm(w(1), w(0), sel), __builtin_amdgcn_perm(w(3), w(2), sel),
                         __builtin_amdgcn_perm(w(5), w(4), sel), __builtin_amdgcn_perm(w(7), w(6), sel)});
        }
      }
    };
    auto stage_end = [&](int b, int buf) {
      if (__builtin_amdgcn_ballot_w64(bad != 0) == 0) return;
      bad_block[buf] = b;                    // every writer writes the same
#pragma unroll
      for (int i = 0; i < VI; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int x = 0; x < E; ++x) vr[i][j][x] = finite_part<FP8>(vr[i][j][x]);
#pragma unroll
      for (int u = NK + NB; u < NU; ++u) stage_unit(u, buf);
    };

    bool marked = false;
    // The scores of block b with block b + 1 (page p) staged on the way; after it the registers take block b + 2.
    auto compute = [&](int b, int p, int p2, auto static_buf) {
      constexpr int buf = decltype(static_buf)::value;
      const int key0 = (t.block0 + b) * KB;
      stage_begin(b + 1, p, buf ^ 1);
      if (!busy || key0 >= hi_max || key0 + KB <= lo_min) {
#pragma unroll
        for (int u = 0; u < NU; ++u) stage_unit(u, buf ^ 1);
        stage_end(b + 1, buf ^ 1);
        if (b + 2 < b1) fetch(b + 2, p2);
        return;
      }
      int gone = 0;
#pragma unroll
      for (int g = 0; g < NG; ++g) gone |= no_page[buf][g] << g;
      gone = uniform(gone);
      const bool partial_keys = gone != 0 || key0 + KB > hi_min || key0 < lo_max;
      if (uniform(bad_block[buf]) == b) {
        // Rare: mark this lane's outputs that see a non-finite value, by reading the block's values again.
        if (!marked)
          for (int i = 0; i < 2 * MW; ++i) marks[i][tid] = 0;
        marked = true;
#pragma unroll 1
        for (int kk = 0; kk < KB; ++kk) {
          const int key = key0 + kk, pk = page_of(a, t, key);
          if (pk < 0) continue;
          const uint8_t* vp = a.v + pk * a.v_page + head_at + (key & mask) * (D * E) + half * (4 * E);
          const bool seen = key >= lo && key < hi;
#pragma unroll 1
          for (int i = 0; i < D / 8 * E; ++i) {          // dwords of this lane's 4-channel groups, 8 channels apart
            constexpr int PER = FP8 ? 4 : 2;
            uint32_t up, down;
            non_finite_signs<FP8>(*reinterpret_cast<const uint32_t*>(vp + (i / E) * (8 * E) + (i % E) * 4), up, down);
            const int bit = i * PER;
            if (!seen) continue;
            marks[bit >> 5][tid] |= up << (bit & 31);
            marks[MW + (bit >> 5)][tid] |= down << (bit & 31);
          }
        }
      }
      f32x16_t s[KB / 32];
      {
        constexpr int AHEAD = 4, NS = KB / 32 * ST;
        u32x4_t f[AHEAD];
        auto read = [&](int x) {
          return *reinterpret_cast<const u32x4_t*>(&ks[buf][k_chunk((x / ST) * 32 + n, (x % ST) * 2 + half)]);
        };
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) f[x] = read(x);
        __builtin_amdgcn_s_setprio(1);        // the wavefront at its matrix instructions goes first (+1.3 %)
        step();
#pragma unroll
        for (int x = 0; x < NS; ++x) {
          const u32x4_t ka = f[x % AHEAD];
          f32x16_t z;
#pragma unroll
          for (int y = 0; y < 16; ++y) z[y] = 0.0f;
          s[x / ST] = mfma32_bf16(ka, q[x % ST], x % ST == 0 ? z : s[x / ST]);
          if (x + AHEAD < NS) f[x % AHEAD] = read(x + AHEAD);
#pragma unroll
          for (int u = x * NU / NS; u < (x + 1) * NU / NS; ++u) stage_unit(u, buf ^ 1);
          step();
        }
      }
      __builtin_amdgcn_s_setprio(0);
      stage_end(b + 1, buf ^ 1);
      if (b + 2 < b1) fetch(b + 2, p2);
      u32x4_t pr[NG] = {};
      if (partial_keys) {
        asm volatile("");        // a branch, not selects paid by every block
#pragma unroll
        for (int kb = 0; kb < KB / 32; ++kb)
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int key = key0 + kb * 32 + 8 * (x >> 2) + 4 * half + (x & 3);
            const bool seen = !((gone >> (kb * 2 + (x >> 3))) & 1) && key >= lo && key < hi;
            s[kb][x] = seen ? s[kb][x] : -__builtin_inff();
          }
      }
      float mx = m;
#pragma unroll
      for (int kb = 0; kb < KB / 32; ++kb)
#pragma unroll
        for (int x = 0; x < 16; ++x) mx = __builtin_fmaxf(mx, s[kb][x]);
      mx = max_across_32(mx);
      if (__builtin_amdgcn_ballot_w64((mx - m) * c > kLazy) != 0) {
        const float f0 = rescale<FP8>(m, mx, c);
        m = mx;
        sum *= f0;
        // (kAcc: taken out of the accumulation registers here and not ahead of the branch)
#pragma unroll
        for (int i = 0; i < DB; ++i) {
          if constexpr (kAcc) asm volatile("" : "+a"(o[i]));
          o[i] *= f0;
          if constexpr (kAcc) asm volatile("" : "+a"(o[i]));
        }
      }
      float mc = exponent_base<FP8>(m, c);
      if (far_scores(mc)) {
        asm volatile("");        // a branch, as above
        const float from = m == kLowest ? 0.0f : m;
#pragma unroll
        for (int kb = 0; kb < KB / 32; ++kb)
#pragma unroll
          for (int x = 0; x < 16; ++x) s[kb][x] -= from;
        mc = -kLift<FP8>;
      }
      // Exponentials of 8 keys (group g) and the product with V, a group behind.
      {
        float p8[8];
        u32x4_t f[DB];
        auto read = [&](int g, int i) {
          return *reinterpret_cast<const u32x4_t*>(&vt[buf][v_chunk(i * 32 + n, g * 2 + half)]);
        };
        auto exps = [&](int g, int j) {
          p8[j] = exp2_fast(__builtin_fmaf(s[g >> 1][(g & 1) * 8 + j], c, -mc));
          sum += p8[j];
          if (j & 1) pr[g][j >> 1] = p_pair<FP8>(p8[j - 1], p8[j]);
        };
#pragma unroll
        for (int i = 0; i < DB; ++i) f[i] = read(0, i);
        step();
#pragma unroll
        for (int j = 0; j < 8; ++j) exps(0, j);
        step();
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int i = 0; i < DB; ++i) {
            const u32x4_t va = f[i];
            o[i] = mfma32_pv<FP8>(va, pr[g], o[i]);
            if (g + 1 < NG) {
              f[i] = read(g + 1, i);
#pragma unroll
              for (int j = i * 8 / DB; j < (i + 1) * 8 / DB; ++j) exps(g + 1, j);
            }
            step();
          }
        }
      }
      if constexpr (kAcc) {
#pragma unroll
        for (int i = 0; i < DB; ++i) asm volatile("" : "+a"(o[i]));
      }
    };

    __syncthreads();                          // the last piece's readers are done
    if (tid < 2) bad_block[tid] = -1;
    int p0 = my_page(b0), p1 = my_page(b0 + 1);    // page numbers come a block ahead of their loads
    fetch(b0, p0);
    __syncthreads();
    stage_begin(b0, p0, 0);
#pragma unroll
    for (int u = 0; u < NU; ++u) stage_unit(u, 0);
    stage_end(b0, 0);
    if (b0 + 1 < b1) fetch(b0 + 1, p1);
    __syncthreads();
    for (int b = b0; b < b1; ++b) {
      const int p2 = my_page(b + 2);
      compute(b, p1, p2, Buffer<0>{});
      p1 = p2;
      __syncthreads();
      if (++b == b1) break;
      const int p3 = my_page(b + 2);
      compute(b, p1, p3, Buffer<1>{});
      p1 = p3;
      __syncthreads();
    }

    if (marked) {
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int bit = i * 16 + x;
          o[i][x] += non_finite_part((marks[bit >> 5][tid] >> (bit & 31)) & 1, (marks[MW + (bit >> 5)][tid] >> (bit & 31)) & 1);
        }
    }
    const float vs = FP8 ? a.v_scale[h * a.scale_stride] : 1.0f;
    const float ll = sum + __shfl_xor(sum, 32, 64);
    const float mm = scaled_max<FP8>(m, c, ll);
    const int tr = wrow + n;
    if (tr >= t.rows) return;
    if (partial >= 0) {
      const int64_t at = (int64_t)partial * BM + tr;
      if (half == 0) l.ml[at] = make_float2(mm, ll);
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *reinterpret_cast<float4*>(l.po + at * D + i * 32 + 8 * x + 4 * half) =
              make_float4(o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]);
    } else {
      const int r = t.row0 + tr;
      const int tok = (int)fastdiv((uint32_t)r, a.div_group), head = h * a.group + r - tok * a.group;
      const float f = 1.0f / ll;
      uint16_t* y = a.out + (t.c0 + tok) * a.o_tok + head * a.o_head;
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *reinterpret_cast<uint2*>(y + i * 32 + 8 * x + 4 * half) =
              make_uint2(bf16_pair(normalised(o[i][4 * x], ll, f, vs), normalised(o[i][4 * x + 1], ll, f, vs)),
                         bf16_pair(normalised(o[i][4 * x + 2], ll, f, vs), normalised(o[i][4 * x + 3], ll, f, vs)));
      if (a.lse && half == 0) a.lse[(int64_t)(t.c0 + tok) * a.q_heads + head] = (mm + __builtin_log2f(ll)) * kLn2;
    }
  });
}

// ---- joining the parts of cut segments ---------------------------------------------------------------

// A row's parts are read by `PARTS` groups of D / 4 lanes (4 channels each) and added in a fixed order; a workgroup
// takes 256 / (D / 4) / PARTS rows at a time of one (slot, head), and rows_grid workgroups share its rows.  Few
// row tiles are cut into many parts (PARTS as large as fits), many row tiles into few (PARTS = 1: no exchange).
// STREAM: shares were planned per sequence, otherwise per slot.  A launch of its own (4 to 12 us): its reads wait for
// every workgroup of the first anyway.
template <int D, int BM, int KB, bool STREAM, int PARTS>
__global__ __launch_bounds__(kThreads) void combine_kernel(AttentionArgs a, Launch l) {
  constexpr int LP = D / 4, GR = kThreads / LP, ROWS = GR / PARTS;
  __shared__ float4 part[PARTS > 1 ? GR : 1][LP];
  __shared__ float2 part_ml[PARTS > 1 ? GR : 1];
  const int tid = threadIdx.x;
  const int rest = blockIdx.x / l.rows_grid;
  const int h = rest % a.kv_heads, slot = rest / a.kv_heads;
  Tile t;
  const int s = wave_search(a.num_seqs, [&](int j) { return first_slot<BM>(a, l, j) <= slot; });
  if (s < 0 || !tile_of<BM, KB>(a, l, s, slot - first_slot<BM>(a, l, s), t)) return;
  const int per = scalar_load(l.plan), all = scalar_load(l.plan + 1);
  int p0, count;
  if (STREAM) {
    int block0;
    sequence_tiles<BM, KB>(a, l, s, block0, count);
    p0 = scalar_load(l.plan + 2 + s) + (slot - first_slot<BM>(a, l, s)) * count;
  } else {
    p0 = scalar_load(l.plan + 2 + slot);
    count = scalar_load(l.plan + 3 + slot) - p0;
  }
  if (count <= 0) return;
  if (per == INT32_MAX) return;              // tiles were kept whole
  const int64_t u0 = (int64_t)h * all + p0, u1 = u0 + count;
  const int w0 = (int)(u0 / per), w1 = (int)((u1 - 1) / per);
  if (w0 == w1) return;
  // the first part is the one its workgroup ended with (the odd slot), the others are the ones theirs began with
  const int64_t first = 2 * (int64_t)w0 + 1;
  const int g = tid / LP, x = tid % LP, pg = g % PARTS;
  for (int row0 = (blockIdx.x % l.rows_grid) * ROWS; row0 < t.rows; row0 += l.rows_grid * ROWS) {
    const int row = row0 + g / PARTS;
    const bool live = row < t.rows;
    float m, sum;
    float4 acc;
    auto start = [&](float2 ml, float4 v) {
      m = ml.x;
      sum = ml.y;
      acc = v;
    };
    auto add = [&](auto keep, float2 ml, float4 v) {
      constexpr bool KEEP = decltype(keep)::value;
      const float mx = __builtin_fmaxf(m, ml.x), f0 = exp2_fast(m - mx), f1 = exp2_fast(ml.x - mx);
      m = mx;
      sum = sum * f0 + ml.y * f1;
      acc.x = weighted<KEEP>(acc.x, f0) + weighted<KEEP>(v.x, f1);
      acc.y = weighted<KEEP>(acc.y, f0) + weighted<KEEP>(v.y, f1);
      acc.z = weighted<KEEP>(acc.z, f0) + weighted<KEEP>(v.z, f1);
      acc.w = weighted<KEEP>(acc.w, f0) + weighted<KEEP>(v.w, f1);
    };
    auto has_nan = [&] {
      const float x4 = acc.x + acc.y + acc.z + acc.w;
      return x4 != x4;
    };
    auto lane_parts = [&](auto keep) {
      start(make_float2(kLowest, 0.0f), make_float4(0, 0, 0, 0));
      for (int w = w0 + pg; w <= w1; w += 4 * PARTS) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int wi = w + i * PARTS;
          const int64_t at = (wi == w0 ? first : 2 * (int64_t)(wi <= w1 ? wi : w1)) * BM + row;
          ml[i] = l.ml[at];
          v[i] = *reinterpret_cast<const float4*>(l.po + at * D + x * 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (w + i * PARTS > w1) continue;
          add(keep, ml[i], v[i]);
        }
      }
      return has_nan();
    };
    if (!live)
      start(make_float2(kLowest, 0.0f), make_float4(0, 0, 0, 0));
    else if (lane_parts(Keep<false>{}))
      lane_parts(Keep<true>{});
    if (PARTS > 1) {
      __syncthreads();
      part[g][x] = acc;
      if (x == 0) part_ml[g] = make_float2(m, sum);
      __syncthreads();
      if (pg != 0) continue;
      auto group_parts = [&](auto keep) {
        start(part_ml[g], part[g][x]);
        for (int i = 1; i < PARTS; ++i) add(keep, part_ml[g + i], part[g + i][x]);
        return has_nan();
      };
      if (group_parts(Keep<false>{})) group_parts(Keep<true>{});
    }
    if (!live) continue;
    const float vs = a.v_scale ? a.v_scale[h * a.scale_stride] : 1.0f;
    const int r = t.row0 + row;
    const int tok = (int)fastdiv((uint32_t)r, a.div_group), head = h * a.group + r - tok * a.group;
    const float f = 1.0f / sum;
    *reinterpret_cast<uint2*>(a.out + (t.c0 + tok) * a.o_tok + head * a.o_head + x * 4) =
        make_uint2(bf16_pair(normalised(acc.x, sum, f, vs), normalised(acc.y, sum, f, vs)),
                   bf16_pair(normalised(acc.z, sum, f, vs), normalised(acc.w, sum, f, vs)));
    if (a.lse && x == 0) a.lse[(int64_t)(t.c0 + tok) * a.q_heads + head] = (m + __builtin_log2f(sum)) * kLn2;
  }
}

// ---- launching ----------------------------------------------------------------------------------------

// One of the two kernels of a call: which rows it takes, its row tile and whether its key axis is cut.
struct Choice {
  bool used;
  int bm, rows_lo, rows_hi;
  int64_t slots;
  bool split;
  int workgroups;
  int rows;                  // rows a tile holds, by the hint
};

struct Choices {
  Choice stream, tile;
};

size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

size_t split_bytes(const Choice& c, int dim) {
  if (!c.used || !c.split) return 0;
  return align16((size_t)(c.slots + 3) * 4) + (size_t)2 * c.workgroups * c.bm * (8 + (size_t)dim * 4);
}

// Threads of a launch, a 32-bit number.
bool fits_a_launch(int64_t workgroups) { return workgroups <= (int64_t)UINT32_MAX / kThreads; }

// Which kernel takes which sequences.  By the hint (or the call's tokens) a sequence has at most `rows` packed rows:
//   up to 32      stream_kernel alone, 16 or 32 rows a tile (8 query heads a group, 4 tokens over 8192 keys: 17 us,
//                 by tile_kernel 26; 16 sequences of 4 tokens, bf16: 47 and 59)
//   more          tile_kernel, and beside it stream_kernel for the sequences that do have few rows; a single
//                 sequence goes to tile_kernel alone
// Both read the real lengths on the device, so a wrong hint costs time only.  The key axis may be cut where row
// tiles are too few to fill the GPU twice (tile_kernel then decides on the device, kCutCost) or, for stream_kernel,
// wherever the plan holds the sequences.
Choices choose(int64_t tokens, int64_t max_q, int64_t num_seqs, int64_t q_heads, int64_t kv_heads, int dim) {
  const int64_t group = q_heads / kv_heads;
  const int64_t rows = (max_q > 0 && max_q < tokens ? max_q : tokens) * group;
  Choices c{};
  auto slots = [&](int bm) { return tokens * group / bm + num_seqs; };
  const int rb = rows <= 16 || (rows > 32 && group <= 16) ? 1 : 2;
  c.stream.used = rows <= 32 || (num_seqs > 1 && group <= 32);
  c.tile.used = rows > 32;
  c.stream.bm = 16 * rb;
  c.stream.rows_hi = c.tile.used ? c.stream.bm : INT32_MAX;
  c.stream.slots = c.tile.used ? num_seqs : slots(c.stream.bm);
  c.stream.split = c.stream.slots <= kMaxSlots;
  c.stream.workgroups = dim == 256 ? 512 : 1024;
  c.stream.rows = (int)(rows < c.stream.bm ? rows : c.stream.bm);
  c.tile.bm = 128;
  c.tile.rows = c.tile.bm;
  c.tile.rows_lo = c.stream.used ? c.stream.bm : 0;
  c.tile.rows_hi = INT32_MAX;
  c.tile.slots = slots(c.tile.bm);
  c.tile.workgroups = dim == 256 ? 256 : 512;
  c.tile.split = c.tile.slots <= kMaxSlots && c.tile.slots * kv_heads < 2 * c.tile.workgroups;
  // (a join has up to a workgroup per row)
  for (Choice* x : {&c.stream, &c.tile}) x->split = x->split && fits_a_launch(x->slots * kv_heads * x->rows);
  return c;
}

template <int D, int BM, int KB, bool STREAM, typename Kernel>
int launch_one(Kernel kernel, const AttentionArgs& a, const Choice& c, int min_blocks, void* workspace, hipStream_t stream) {
  Launch l{};
  l.slots = (int32_t)c.slots;
  l.rows_lo = c.rows_lo;
  l.rows_hi = c.rows_hi;
  l.min_blocks = min_blocks;
  // nothing to cut where the table holds no more keys than the smallest share, or where block
  // numbers could pass 31 bits
  const int64_t cap = (((int64_t)a.table_width << a.page_shift) + KB - 1) / KB;
  l.split = c.split && cap > min_blocks &&
            plan_fits(STREAM, c.slots, a.num_seqs, (int64_t)a.tokens * a.group, c.rows_hi, BM, cap, a.kv_heads, c.workgroups);
  l.workgroups = c.workgroups;
  int64_t grid = c.slots * a.kv_heads;
  if (l.split) {
    // (tile_kernel may keep its tiles whole: then one workgroup each, handed out as they come)
    if (STREAM || grid < c.workgroups) grid = c.workgroups;
    char* p = static_cast<char*>(workspace);
    l.plan = reinterpret_cast<int32_t*>(p);
    l.ml = reinterpret_cast<float2*>(p + align16((size_t)(c.slots + 3) * 4));
    l.po = reinterpret_cast<float*>(l.ml + (size_t)2 * c.workgroups * BM);
  }
  kernel<<<(unsigned)grid, kThreads, 0, stream>>>(a, l);
  if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
  if (l.split) {
    constexpr int kRows = kThreads / (D / 4);            // rows a workgroup holds at once, a part each
    const int64_t segments = c.slots * a.kv_heads;
    if (segments * c.rows < 1024) {
      l.rows_grid = c.rows;
      combine_kernel<D, BM, KB, STREAM, kRows><<<(unsigned)(segments * l.rows_grid), kThreads, 0, stream>>>(a, l);
    } else {
      l.rows_grid = (c.rows + kRows - 1) / kRows;
      combine_kernel<D, BM, KB, STREAM, 1><<<(unsigned)(segments * l.rows_grid), kThreads, 0, stream>>>(a, l);
    }
    if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
  }
  return NVFP4_OK;
}

template <int D, bool FP8>
int launch_dim(const AttentionArgs& a, const Choices& c, void* workspace, hipStream_t stream) {
  // smallest shares: 2 blocks of 128 keys (a captured call of one token over 4096 keys 12.1 us, 1 block 11.2, 4 blocks
  // 13.4; over 16384 keys 17.6, 22.7 and 17.0) and 4 of 64 keys
  if (c.stream.used) {
    const int st = c.stream.bm == 16
        ? launch_one<D, 16, kStreamBlock, true>(stream_kernel<D, FP8, 1>, a, c.stream, 2, workspace, stream)
        : launch_one<D, 32, kStreamBlock, true>(stream_kernel<D, FP8, 2>, a, c.stream, 2, workspace, stream);
    if (st != NVFP4_OK) return st;
  }
  if (c.tile.used) return launch_one<D, 128, kTileBlock, false>(tile_kernel<D, FP8>, a, c.tile, 256 / kTileBlock, workspace, stream);
  return NVFP4_OK;
}

}  // namespace

size_t paged_attention_workspace_bytes(int64_t tokens, int64_t max_q, int64_t num_seqs, int64_t q_heads,
                                       int64_t kv_heads, int head_dim) {
  const Choices c = choose(tokens, max_q, num_seqs, q_heads, kv_heads, head_dim);
  const size_t s = split_bytes(c.stream, head_dim), t = split_bytes(c.tile, head_dim);
  return s > t ? s : t;
}

int launch_paged_attention(const AttentionArgs& a, int64_t max_q, int head_dim, void* workspace, hipStream_t stream) {
  const Choices c = choose(a.tokens, max_q, a.num_seqs, a.q_heads, a.kv_heads, head_dim);
  for (const Choice& x : {c.stream, c.tile})           // before anything is enqueued
    if (x.used && !fits_a_launch(x.slots * a.kv_heads)) return NVFP4_ERR_UNSUPPORTED;
  const bool fp8 = a.k_scale != nullptr;
  switch (head_dim) {
    case 64: return fp8 ? launch_dim<64, true>(a, c, workspace, stream) : launch_dim<64, false>(a, c, workspace, stream);
    case 128: return fp8 ? launch_dim<128, true>(a, c, workspace, stream) : launch_dim<128, false>(a, c, workspace, stream);
    default: return fp8 ? launch_dim<256, true>(a, c, workspace, stream) : launch_dim<256, false>(a, c, workspace, stream);
  }
}

}  // namespace nvfp4
