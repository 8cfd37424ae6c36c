// Attention of a tree of drafted tokens over a KV cache, on tcgen05.
//
// Several drafted tokens of a sequence, arranged as a tree, are verified in one pass over its cache
// (ONNX Runtime packed-QSA analysis, "Code analysis" 2: multi-token verification).  The cache already
// holds the drafts as its last tokens: with base = kv_len - q_len, token i sees slot t when t < base,
// or when t < kv_len and bit (t - base) of its 64-bit mask is set:
//     o_i = sum_t softmax_t(scale * q_i . k_t) v_t     over the slots t that token i sees.
//
// Rows.  The G query heads of a KV head share its keys, so row r = (i - i0) * G + g of a 128-row "slot"
// is token i, head g of the group; a slot holds tps = floor(128 / G) tokens.  Q lands in that order
// straight from [B, n_q, Hq, D] through a 5-D TMA box (64, G, tps, 1, 1).
//   PAIR  (n_q > tps): the CTA's two slots are two row slots; every staged K/V tile feeds 256 rows.
//         More than 256 rows are n_rb row blocks, run by neighbouring CTAs over the same tiles at
//         the same time, so the cache crosses HBM once and the other blocks hit L2.
//   !PAIR (n_q <= tps): the two slots hold the same rows and take alternate key tiles; their softmax
//         states are joined in the epilogue.  One slot alone would leave the softmax of a tile
//         and its two MMAs in series (~2300 cycles a tile against ~1450 of HBM time at 8 bits).
//         So does a PAIR kernel over a coded cache with a sequence whose drafts fit one slot (MIXED): of up to 25
//         drafts (b8 g7 t10007 INT8), 18 in every sequence took 77 us with one slot idle and take 59, one 67 and 56.
//
// Work.  The (sequence, KV head, 128-key tile) triples in that order are one line of W tiles, cut into
// equal contiguous ranges, one per CTA (one per n_rb neighbouring CTAs): ragged lengths leave no CTA
// with less to read, whatever Tmax is.  A range covers pieces of items (sequence, KV head); a piece
// that is a whole item is finished here, another leaves a normalised partial in the workspace and
// tree_join merges an item's partials in tile order (no atomics: results repeat bit for bit).
//
// Pipeline, as the prefill's: S = Q K^T in TMEM, one thread per row for the softmax, P (bf16; f16 for coded
// caches) over S, O += P V; unit ring of MMA-ready K and V tiles in consumption order.  Coded caches (E4M3, INT8, INT4)
// land raw in a ring of their own and a fourth warpgroup widens them to f16, which is exact for
// every code (one instruction per two E4M3 codes, five per four INT8 codes; bf16 took five and eight);
// the queries follow as f16 times a power of two, one for all of a piece's rows but those far below its largest,
// which get their own (a padded draft's query may be anything, and is nobody else's business).  The K scale
// multiplies the fp32 score and the V scale the fp32 weight before its one rounding to f16, so no scale is
// rounded.  A row's weights are taken relative to its largest weight times V scale, max_t (y_t + log2
// |v_scale_t|), not to its largest weight, and from a reference REF_DROP powers of two below it, in f16's upper
// range: the row's largest product is 2^3 to 2^15, so products down to 2^-17 of it keep f16's full precision
// whatever the scales and those below are off by at most 2^-28 of it.  (With the largest at 2^-8 to 2^8, 128K flat
// tokens behind a sink were off by up to half of their part.)
//
// Masked places.  Slots past kv_len and drafts no token sees are never used.  A draft that some tokens
// see may hold anything too: its non-finite V elements enter the MMA as zeros (0 * NaN would reach
// the rows that do not see it) and the epilogue adds them back to the rows that do.
#pragma once

#include <type_traits>

#include "decode_int.cuh"
#include "device_ext.cuh"

namespace attn {

struct TreeParams {
  int B, Hq, Hkv, G, Tmax, n_q;
  int tps;       // tokens per 128-row slot
  int n_rb;      // row blocks (CTAs that share a range of tiles)
  int n_groups;  // ranges (grid = n_groups * n_rb)
  float scale_log2;
  const int* kv_lens;       // [B]
  const int* q_lens;        // [B] or null (n_q)
  const long long* mask;    // [B, n_q]
  const void* v;            // the V cache again, for the epilogue's non-finite drafts
  const float* k_scale;     // coded caches: [pages, page_size, Hkv]
  const float* v_scale;
  const int* page_table;    // [B, max_pages] or null (one page of Tmax tokens per sequence)
  int max_pages, page_size, num_pages;
  float* part_o;            // [n_groups * n_rb * 2, D, rows] normalised partials
  float* part_lse;          // [n_groups * n_rb * 2, rows] their log2-domain log-sum-exp
  __nv_bfloat16* o;         // [B, n_q, Hq, D]
  float* lse;               // [B, n_q, Hq] or null
};

// Ranges an item can be cut into: the launch has one CTA per processor, of which there are fewer.
static constexpr int kTreeMaxRanges = 256;

enum TreeKv { TREE_BF16 = 0, TREE_FP8 = 1, TREE_INT8 = 2, TREE_INT4 = 3 };

__device__ __forceinline__ int tree_len(const TreeParams& p, int b) {
  const int len = __ldg(p.kv_lens + b);
  return len < 0 ? 0 : (len > p.Tmax ? p.Tmax : len);
}
__device__ __forceinline__ int tree_qlen(const TreeParams& p, int b) {
  if (!p.q_lens) return p.n_q;
  const int n = __ldg(p.q_lens + b);
  return n < 0 ? 0 : (n > p.n_q ? p.n_q : n);
}
// Key tiles of one KV head of sequence b (none when it drafts nothing).
__device__ __forceinline__ int tree_tiles(const TreeParams& p, int b) {
  const int qn = tree_qlen(p, b), n = (tree_len(p, b) + 127) >> 7;  // two loads at once, not one after the other
  return qn > 0 ? n : 0;
}

// Pool page of token tok of sequence b, -1 (never dereferenced: TMA fills zeros, scales read as 0) for a
// table entry outside the pool, which is reported.
__device__ __forceinline__ int tree_page(const TreeParams& p, int b, int tok) {
  if (!p.page_table) return b;
  const int pg = __ldg(p.page_table + (long long)b * p.max_pages + tok / p.page_size);
  if (pg >= 0 && pg < p.num_pages) return pg;
  record_arg_error(ATTN_DEV_BAD_PAGE, SITE_TR_PAGE);
  return -1;
}
__device__ __forceinline__ int tree_page_off(const TreeParams& p, int tok) {
  return p.page_table ? tok % p.page_size : tok;
}

// Where the range of group g starts: floor(g * W / ng).
__device__ __forceinline__ int tree_range(int g, int W, int ng) { return (int)((long long)g * W / ng); }

struct TreePiece {
  int b, kvh, t0, n;  // tiles t0 .. t0 + n - 1 of (sequence, KV head)
  int len, qn;        // the sequence's cache length and drafted tokens
  int which;          // 0: the first piece of this CTA's range, 1: a later one (names its partial)
  bool whole;         // every tile of the item
  int idx, joins;     // softmax warps: earlier pieces, those whose tiles the slots took in turn
};

// The pieces of a CTA's range, in order; every role walks its own copy.
struct TreeWalk {
  int left, b, kvh, tile, idx;
  int len, qn, tiles;
  __device__ __forceinline__ void load(const TreeParams& p) {
    len = tree_len(p, b);
    qn = tree_qlen(p, b);
    tiles = qn > 0 ? (len + 127) >> 7 : 0;
  }
  // s: {tiles of the range, first sequence, tile offset within that sequence's Hkv * tiles}
  __device__ __forceinline__ void init(const TreeParams& p, const int* s) {
    left = s[0];
    b = s[1];
    idx = 0;
    kvh = tile = 0;
    if (left > 0) {
      load(p);
      kvh = s[2] / tiles;
      tile = s[2] - kvh * tiles;
    }
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreePiece& out) {
    if (left <= 0) return false;
    while (kvh == p.Hkv || tiles == 0) {  // left > 0: a later sequence has tiles
      ++b;
      kvh = 0;
      load(p);
    }
    const int n = min(tiles - tile, left);
    out.b = b;
    out.kvh = kvh;
    out.t0 = tile;
    out.n = n;
    out.len = len;
    out.qn = qn;
    out.which = idx > 0;
    out.idx = idx;
    out.whole = n == tiles;
    ++idx;
    left -= n;
    tile += n;
    if (tile == tiles) {
      tile = 0;
      ++kvh;
    }
    return true;
  }
};

// One warp: total tiles, this group's range, and the sequence it starts in -> s[0..2].
__device__ __forceinline__ void tree_find_range(const TreeParams& p, int g, int lane, int* s) {
  int total = 0;
  for (int b = lane; b < p.B; b += 32) total += tree_tiles(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int W = total * p.Hkv;
  const int ng = min(p.n_groups, W);
  int left = 0, start = 0;
  if (g < ng) {
    start = tree_range(g, W, ng);
    left = tree_range(g + 1, W, ng) - start;
  }
  int b0 = 0, off = 0, before = 0;
  if (left > 0) {
    for (int c = 0; c < p.B; c += 32) {
      const int b = c + lane;
      const int n = (b < p.B ? tree_tiles(p, b) : 0) * p.Hkv;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > start);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b0 = c + src;
        off = start - (before + __shfl_sync(0xffffffffu, incl - n, src));
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (lane == 0) {
    s[0] = left;
    s[1] = b0;
    s[2] = off;
  }
}

template <int KIND, int D, bool PAIR>
struct TreeCfg {
  static constexpr bool CODED = KIND != TREE_BF16;
  // A sequence of fewer drafts than n_q may need one row slot only.  bf16 has no shared memory left for the join.
  static constexpr bool MIXED = PAIR && CODED;
  static constexpr int BOX_BYTES = 128 * 128;  // 128 rows x 64 bf16
  static constexpr int NBOX = D / 64;
  static constexpr int TILE_BYTES = NBOX * BOX_BYTES;
  static constexpr int NQ = PAIR ? 2 : 1;  // Q slots in shared memory
  // MMA-ready units in flight, raw units in flight (coded caches), scale tiles in flight.
  static constexpr int NU = D == 64 ? 6 : (CODED ? (PAIR ? 3 : 4) : 5);
  static constexpr int RAW_BYTES = 128 * (KIND == TREE_INT4 ? D / 2 : D);
  static constexpr int NR = CODED ? (KIND == TREE_INT4 ? 6 : 3) : 0;
  static constexpr int NS = CODED ? 4 : 0;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_U = OFF_Q + NQ * TILE_BYTES;
  static constexpr int OFF_RAW = OFF_U + NU * TILE_BYTES;
  static constexpr int OFF_SC = OFF_RAW + NR * RAW_BYTES;      // [NS][3][128] floats
  static constexpr int OFF_ML = OFF_SC + NS * (1536 + 32);            // [2 slots][128] (max, sum) of the halves
  static constexpr int OFF_WALK = OFF_ML + (PAIR && !MIXED ? 0 : 2048);  // [8] walks, [8] pieces of the softmax warps
  static constexpr int OFF_BAR = OFF_WALK + 8 * (int)(sizeof(TreeWalk) + sizeof(TreePiece));
  static constexpr int N_BARS = 3 + 2 * NU + 2 * NR + 2 * NS + 2 + 2 + 2 + 2 + 1 + 1;
  static constexpr int OFF_ROWF = OFF_BAR + N_BARS * 8 + 72;  // + walk start, flags; [2 pieces][NQ][128] row factors
  static constexpr int SMEM_BYTES = OFF_ROWF + (CODED ? 2 * NQ * 512 : 0) + 1024;  // + alignment slack
  static constexpr int THREADS = CODED ? 512 : 384;
  // Register split: the softmax holds a row's 128 scores (bf16) or half of them (coded caches, of whose 512
  // threads a launch has 128 registers each), and the other warpgroups give up what that takes.  The sum
  // never exceeds what the launch holds (checked on the host before the first launch).  The coded kernels spill one
  // 4-byte value (-Xptxas -v: one store, one or five loads), the bf16 ones nothing; more would show: next to 200 KB of
  // shared memory there is hardly any L1, and a reload takes some 300 cycles.
  static constexpr int REGS_CTRL = CODED ? 96 : 104;  // the MMA issuer of two row slots needs them
  static constexpr int REGS_CONV = 96;
  static constexpr int REGS_SOFTMAX = CODED ? 160 : 200;
  static constexpr int REGS_TOTAL = (REGS_CTRL + (CODED ? REGS_CONV : 0) + 2 * REGS_SOFTMAX) * 128;
  static constexpr uint32_t EXP_MASK = CODED ? 0x7c00u : 0x7f80u;  // exponent field of an MMA operand
  // Scales of a tile: K (times all score factors), V, log2 |V|, then from either scale warp, for its 64 tokens, the
  // largest and smallest of K's and of the logarithms.
  static constexpr int SC_BYTES = 3 * 512 + 32;
  static constexpr uint32_t TMEM_COLS = 512;
  // A row's reference may lag its maximum by RESCALE_THRESHOLD and lies REF_DROP below (an upper bound of) it:
  // products reach 2^(4 + 11), of f16's 65504.  A bound may exceed the maximum by REF_SLACK, so the largest
  // product is at least 2^(11 - 8).  A sum of weights stays below 2^(15 + LOG_MIN's 80) a token.  Measured side by side
  // (b8 n16 t32768 FP8, INT8, INT4 on N(0, 1) values): 203, 219, 215 us with a threshold of 8, a drop of 7 and a slack of
  // 8 (floor 2^-24); 205, 219, 215 so (2^-28); 211, 225, 223 with a slack of 7, which sends more tiles column by column.
  // Where K scales differ so much that every tile goes that way (over 2^4) it takes 246, 259, 251 us, not 198, 214, 206.
  static constexpr float RESCALE_THRESHOLD = CODED ? 4.0f : 8.0f;
  static constexpr float REF_DROP = 11.0f, REF_SLACK = 8.0f;
  static constexpr float LOG_MIN = -80.0f, LOG_MAX = 100.0f;  // of log2 |V scale|
  static constexpr int ROWS = PAIR ? 256 : 128;  // rows of a partial
};

// Unit order within a piece of n tiles (units K(0..n-1), V(0..n-1); 2n in all).
//   PAIR: K0 V0 K1 V1 ...            !PAIR: K0 K1 V0 K2 V1 K3 V2 ...
template <bool PAIR>
__device__ __forceinline__ int tree_v_unit(int j, int n) {
  return PAIR ? 2 * j + 1 : min(j + 2, n) + j;
}

// 16 raw codes -> 32 bytes of f16 (two 16-byte chunks), exact.  INT4 groups of eight come out in the order of
// i4x8_to_f16_paired; the queries take the same order, and the epilogue undoes it for V.
template <int KIND>
__device__ __forceinline__ void tree_widen(const uint32_t (&w)[4], uint4& lo, uint4& hi) {
  uint32_t r[8];
  if constexpr (KIND == TREE_FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[2 * i] = e4m3x2_to_f16x2((uint16_t)(w[i] & 0xffffu));
      r[2 * i + 1] = e4m3x2_to_f16x2((uint16_t)(w[i] >> 16));
    }
  } else if constexpr (KIND == TREE_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) i8x4_to_f16(w[i], r[2 * i], r[2 * i + 1]);
  } else {
    i4x8_to_f16_paired(w[0], r);
    i4x8_to_f16_paired(w[1], r + 4);
  }
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
}

// Where element d of a group of eight stands in the paired order (0, 4, 1, 5, 2, 6, 3, 7).
template <int KIND>
__host__ __device__ constexpr int tree_place(int d) {
  return KIND == TREE_INT4 ? (d & ~7) | ((d & 3) << 1) | ((d >> 2) & 1) : d;
}

// Non-finite elements of a packed pair (exponent field EXP all ones) set to zero; true if there was one.
template <uint32_t EXP>
__device__ __forceinline__ bool drop_nonfinite(uint32_t& w) {
  bool bad = false;
  if ((w & EXP) == EXP) {
    w &= 0xffff0000u;
    bad = true;
  }
  if ((w & (EXP << 16)) == (EXP << 16)) {
    w &= 0x0000ffffu;
    bad = true;
  }
  return bad;
}

// Row r of an MMA-ready V tile: zeros when drop, else its non-finite elements set to zero (true if any).
template <int NBOX, uint32_t EXP>
__device__ __forceinline__ bool tree_scrub_row(uint8_t* tile, int r, bool drop) {
  bool odd = false;
#pragma unroll 1
  for (int x = 0; x < NBOX * 8; ++x) {
    uint4* q4 = reinterpret_cast<uint4*>(tile + (x >> 3) * (128 * 128) + sw128_offset(r, x & 7));
    uint4 v4 = make_uint4(0u, 0u, 0u, 0u);
    bool bad = drop;
    if (!drop) {
      v4 = *q4;
      bad |= drop_nonfinite<EXP>(v4.x);
      bad |= drop_nonfinite<EXP>(v4.y);
      bad |= drop_nonfinite<EXP>(v4.z);
      bad |= drop_nonfinite<EXP>(v4.w);
      odd |= bad;
    }
    if (bad) *q4 = v4;
  }
  return odd;
}

// One V element of the cache as float (the epilogue's slow path).
template <int KIND, int D>
__device__ __forceinline__ float tree_v_value(const TreeParams& p, long long row, int d) {
  if constexpr (KIND == TREE_BF16) {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v)[row * D + d]);
  } else {
    float c;
    if constexpr (KIND == TREE_INT8) {
      c = (float)reinterpret_cast<const int8_t*>(p.v)[row * D + d];
    } else if constexpr (KIND == TREE_INT4) {
      const int x = reinterpret_cast<const uint8_t*>(p.v)[row * (D / 2) + (d >> 1)];
      const int n = (d & 1) ? x >> 4 : x & 15;
      c = (float)(n >= 8 ? n - 16 : n);
    } else {
      const uint32_t h = e4m3x2_to_f16x2(reinterpret_cast<const uint8_t*>(p.v)[row * D + d]);
      c = __low2float(*reinterpret_cast<const __half2*>(&h));
    }
    return c * p.v_scale[row];
  }
}

// Every draft that some token of sequence b sees, as a 64-bit set (warp-collective).
__device__ __forceinline__ unsigned long long tree_seen_any(const TreeParams& p, int b, int qn, int lane) {
  const long long* m = p.mask + (long long)b * p.n_q;
  unsigned long long x = 0;
  if (lane < qn) x |= (unsigned long long)__ldg(m + lane);
  if (lane + 32 < qn) x |= (unsigned long long)__ldg(m + lane + 32);
  const uint32_t lo = __reduce_or_sync(0xffffffffu, (uint32_t)x);
  const uint32_t hi = __reduce_or_sync(0xffffffffu, (uint32_t)(x >> 32));
  return ((unsigned long long)hi << 32) | lo;
}

__device__ __forceinline__ unsigned long long tree_low_bits(int n) {
  return n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// Columns col .. col + 31 of the tile at kv0 that a row sees: slots below base, and drafts in m.
__device__ __forceinline__ uint32_t tree_seen_word(int col, int kv0, int base, unsigned long long m) {
  const int pre = base - kv0 - col;  // leading columns of this word that are below base
  uint32_t x = pre <= 0 ? 0u : (pre >= 32 ? ~0u : (1u << pre) - 1u);
  const int q = -pre;  // the draft that column 0 of the word would be
  if (q > -32 && q < 64) x |= q < 0 ? (uint32_t)(m << -q) : (uint32_t)(m >> q);
  return x;
}

template <int KIND, int D, bool PAIR>
__global__ void __launch_bounds__((TreeCfg<KIND, D, PAIR>::THREADS), 1)
    decode_tree_sm100(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const TreeParams p) {
  using C = TreeCfg<KIND, D, PAIR>;
  constexpr bool CODED = C::CODED;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  // Phases: q_*, o_* complete once per piece (qi); u_full / u_empty once per use of a unit (u);
  // raw_* once per raw unit, sc_* once per tile, s_full / p_full once per tile of their slot.
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* q_raw = bars + 2;  // coded caches: bf16 queries landed (q_full: they are f16)
  uint64_t* u_full = bars + 3;
  uint64_t* u_empty = u_full + C::NU;
  uint64_t* raw_full = u_empty + C::NU;
  uint64_t* raw_empty = raw_full + C::NR;
  uint64_t* sc_full = raw_empty + C::NR;
  uint64_t* sc_empty = sc_full + C::NS;
  uint64_t* s_full = sc_empty + C::NS;  // [2]
  uint64_t* p_full = s_full + 2;        // [2]
  uint64_t* o_full = p_full + 2;
  uint64_t* o_empty = o_full + 1;
  uint64_t* ml_full = o_empty + 1;      // the halves' (max, sum) are in shared memory (8 warps; once per joined piece)
  uint64_t* ml_empty = ml_full + 1;     // ... and have been read
  uint64_t* drain = ml_empty + 1;
  uint64_t* q_meet = drain + 1;         // the converter warps' q_max are in shared memory
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(q_meet + 1);
  int* walk0 = reinterpret_cast<int*>(tmem_holder + 1);   // [3]
  // odd_piece[i & 7] = i + 1 when piece i holds a non-finite draft V.  Whoever finds one runs at most a ring ahead
  // of the epilogue that asks (NU <= 6 units, two or more a piece; NS = 4 tiles of scales): eight entries.
  int* odd_piece = walk0 + 3;
  uint32_t* q_max = reinterpret_cast<uint32_t*>(odd_piece + 8);  // [4] largest |q| (bf16 bits) per converter warp
  float* q_down = reinterpret_cast<float*>(q_max + 4);  // what undoes the queries' power of two
  // What takes a row's scores to that power, by piece parity: its readers are done with piece i before the MMA has done
  // the scores of piece i + 1 (every P of i comes first), which the queries of piece i + 2 wait for.
  float* row_factor = reinterpret_cast<float*>(smem + C::OFF_ROWF);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rb = (int)blockIdx.x % p.n_rb;
  // Whether the two slots hold different rows of this piece (else they take its tiles in turn).
  auto paired = [&](const TreePiece& it) -> bool {
    return PAIR && (!C::MIXED || it.qn > (rb * 2 + 1) * p.tps);
  };
  grid_launch_dependents();  // tree_join's CTAs find room as this kernel's leave

  if (threadIdx.x == 0) {
    mbar_init(q_full, CODED ? 4 : 1);
    mbar_init(q_raw, 1);
    mbar_init(q_empty, CODED ? 3 : 1);  // the MMA is done with the queries, and the scale warps with q_down
    for (int i = 0; i < C::NU; ++i) {
      mbar_init(&u_full[i], CODED ? 4 : 1);  // converter warps, or the producer's expect_tx
      mbar_init(&u_empty[i], 1);
    }
    for (int i = 0; i < C::NR; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&sc_full[i], 2);
      mbar_init(&sc_empty[i], PAIR ? 8 : 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
    }
    mbar_init(o_full, 1);
    mbar_init(o_empty, 8);
    mbar_init(ml_full, 8);
    mbar_init(ml_empty, 8);
    mbar_init(drain, 1);
    mbar_init(q_meet, 4);
    for (int i = 0; i < 8; ++i) odd_piece[i] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 2) tree_find_range(p, (int)blockIdx.x / p.n_rb, lane, walk0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    regs_dec<C::REGS_CTRL>();
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      // A tile is read by the n_rb CTAs of its group at about the same time and never again.
      const uint64_t pol = l2_policy_evict_first();
      const uint32_t q_box = (uint32_t)(p.tps * p.G) * 128u;
      int u = 0, qi = 0;  // units and pieces' queries asked for
      bool ok = true;
      auto load = [&](const CUtensorMap* tm, const TreePiece& it, int j) -> bool {
        const int tok = (it.t0 + j) * 128;
        const int pg = tree_page(p, it.b, tok), off = tree_page_off(p, tok);
        if constexpr (CODED) {
          const int st = u % C::NR;
          if (!mbar_wait<true>(&raw_empty[st], ((u / C::NR) & 1) ^ 1, SITE_TR_LOAD)) return false;
          mbar_arrive_expect_tx(&raw_full[st], C::RAW_BYTES);
          tma_load_4d_hint(smem + C::OFF_RAW + st * C::RAW_BYTES, tm, &raw_full[st], 0, it.kvh, off, pg, pol);
        } else {
          const int st = u % C::NU;
          if (!mbar_wait<true>(&u_empty[st], ((u / C::NU) & 1) ^ 1, SITE_TR_LOAD)) return false;
          mbar_arrive_expect_tx(&u_full[st], C::TILE_BYTES);
          for (int bx = 0; bx < C::NBOX; ++bx)
            tma_load_4d_hint(smem + C::OFF_U + st * C::TILE_BYTES + bx * C::BOX_BYTES, tm, &u_full[st], bx * 64,
                             it.kvh, off, pg, pol);
        }
        ++u;
        return true;
      };
      TreeWalk w;
      TreePiece it;
      w.init(p, walk0);
      while (ok && w.next(p, it)) {
        if (qi > 0 && !(ok = mbar_wait<true>(q_empty, (qi - 1) & 1, SITE_TR_LOAD))) break;
        uint64_t* q_land = CODED ? q_raw : q_full;
        mbar_arrive_expect_tx(q_land, C::NQ * C::NBOX * q_box);
        for (int s = 0; s < C::NQ; ++s)
          for (int bx = 0; bx < C::NBOX; ++bx)
            tma_load_5d(smem + C::OFF_Q + s * C::TILE_BYTES + bx * C::BOX_BYTES, &tmQ, q_land, bx * 64, 0,
                        (rb * C::NQ + s) * p.tps, it.kvh, it.b);
        ++qi;
        if (paired(it)) {
          for (int j = 0; j < it.n && ok; ++j) ok = load(&tmK, it, j) && load(&tmV, it, j);
        } else {
          ok = load(&tmK, it, 0) && (it.n < 2 || load(&tmK, it, 1));
          for (int j = 0; j < it.n && ok; ++j) ok = load(&tmV, it, j) && (j + 2 >= it.n || load(&tmK, it, j + 2));
        }
      }
      // Let every copy asked for land before the CTA's shared memory is released, whatever became of its readers: they
      // may have given up (another CTA's wait ran out) while this warp had nothing left to wait for.  One loop for the
      // queries (its first turn) and the units: more code costs the other roles (b4 n64 64K-128K bf16: 464 us so, 490
      // with two loops).
      constexpr int N = CODED ? C::NR : C::NU;
      const int u0 = max(u - N, 0);
#pragma unroll 1
      for (int t = u0 - (qi > 0); t < u; ++t) {
        const bool is_q = t < u0;
        uint64_t* bar = is_q ? (CODED ? q_raw : q_full) : (CODED ? raw_full : u_full) + t % N;
        mbar_wait_drain<true>(bar, (is_q ? qi - 1 : t / N) & 1, SITE_TR_DRAIN);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    regs_dec<C::REGS_CTRL>();
    {
      constexpr uint32_t idesc_qk = make_idesc_f16(128, 128, false, false, !CODED);
      constexpr uint32_t idesc_pv = make_idesc_f16(128, D, false, true, !CODED);
      constexpr uint32_t HI = sdesc_sw128_hi(1024);
      const uint32_t q_lo = sdesc_sw128_lo(smem_u32(smem + C::OFF_Q), 16);
      const uint32_t k_lo = sdesc_sw128_lo(smem_u32(smem + C::OFF_U), 16);
      const uint32_t v_lo = sdesc_sw128_lo(smem_u32(smem + C::OFF_U), C::BOX_BYTES);
      auto issue_qk = [&](int s, int qs, int st) {
        const uint32_t a0 = q_lo + ((qs * C::TILE_BYTES) >> 4), b0 = k_lo + ((st * C::TILE_BYTES) >> 4);
        const uint32_t d = tmem + s * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::BOX_BYTES + (kk & 3) * 32) >> 4;
          mma_ss_elect(d, sdesc_join(a0 + off, HI), sdesc_join(b0 + off, HI), idesc_qk, kk > 0);
        }
      };
      auto issue_pv = [&](int s, int st, bool acc) {
        const uint32_t b0 = v_lo + ((st * C::TILE_BYTES) >> 4);
        const uint32_t d = tmem + 256 + s * D, a = tmem + s * 128;
#pragma unroll
        for (int kk = 0; kk < 128 / 16; ++kk)
          mma_ts_elect(d, a + kk * 8, sdesc_join(b0 + ((kk * 16 * 128) >> 4), HI), idesc_pv,
                       (acc || kk > 0) ? 1u : 0u);
      };
      int u = 0, qi = 0, c0 = 0, c1 = 0;  // units consumed, pieces, tiles of each slot
      bool ok = true;
      auto wait_unit = [&](int& st) -> bool {
        st = u % C::NU;
        const bool r = mbar_wait_warp<true>(&u_full[st], (u / C::NU) & 1, SITE_TR_MMA_U);
        ++u;
        return r;
      };
      TreeWalk w;
      TreePiece it;
      w.init(p, walk0);
      while (ok && w.next(p, it)) {
        const int n = it.n;
        int st = 0;
        if (!(ok = mbar_wait_warp<true>(q_full, qi & 1, SITE_TR_MMA_Q))) break;
        if (paired(it)) {
          if (!(ok = wait_unit(st))) break;
          tc_fence_after();
          // S(0) of this piece overwrites S/P regions the previous piece's PVs read: those were
          // issued earlier by this warp and the tensor pipe executes in order.
          issue_qk(0, 0, st);
          mma_commit_elect(&s_full[0]);
          issue_qk(1, 1, st);
          mma_commit_elect(&s_full[1]);
          mma_commit_elect(&u_empty[st]);
          if (n == 1) mma_commit_elect(q_empty);
          for (int j = 0; j < n; ++j) {
            const bool more = j + 1 < n;
            int sv, sk = 0;
            if (!(ok = wait_unit(sv))) break;
            if (!(ok = mbar_wait_warp<true>(&p_full[0], c0 & 1, SITE_TR_MMA_P))) break;
            if (j == 0 && qi > 0 && !(ok = mbar_wait_warp<true>(o_empty, (qi - 1) & 1, SITE_TR_MMA_P))) break;
            tc_fence_after();
            issue_pv(0, sv, j > 0);
            if (more) {
              if (!(ok = wait_unit(sk))) break;
              tc_fence_after();
              issue_qk(0, 0, sk);
              mma_commit_elect(&s_full[0]);
            }
            if (!(ok = mbar_wait_warp<true>(&p_full[1], c1 & 1, SITE_TR_MMA_P))) break;
            tc_fence_after();
            issue_pv(1, sv, j > 0);
            mma_commit_elect(&u_empty[sv]);
            if (more) {
              issue_qk(1, 1, sk);
              mma_commit_elect(&s_full[1]);
              mma_commit_elect(&u_empty[sk]);
              if (j + 2 == n) mma_commit_elect(q_empty);
            }
            ++c0;
            ++c1;
          }
        } else {
          for (int s = 0; s < 2 && s < n; ++s) {
            if (!(ok = wait_unit(st))) break;
            tc_fence_after();
            issue_qk(s, 0, st);
            mma_commit_elect(&s_full[s]);
            mma_commit_elect(&u_empty[st]);
          }
          if (!ok) break;
          if (n <= 2) mma_commit_elect(q_empty);
          for (int j = 0; j < n; ++j) {
            const int s = j & 1;
            if (!(ok = wait_unit(st))) break;
            if (!(ok = mbar_wait_warp<true>(&p_full[s], (s ? c1 : c0) & 1, SITE_TR_MMA_P))) break;
            if (j == 0 && qi > 0 && !(ok = mbar_wait_warp<true>(o_empty, (qi - 1) & 1, SITE_TR_MMA_P))) break;
            tc_fence_after();
            issue_pv(s, st, j > 1);
            mma_commit_elect(&u_empty[st]);
            if (j + 2 < n) {
              if (!(ok = wait_unit(st))) break;
              tc_fence_after();
              issue_qk(s, 0, st);
              mma_commit_elect(&s_full[s]);
              mma_commit_elect(&u_empty[st]);
              if (j + 3 == n) mma_commit_elect(q_empty);
            }
            if (s) ++c1;
            else ++c0;
          }
        }
        if (!ok) break;
        mma_commit_elect(o_full);
        ++qi;
      }
      // Drain: every MMA issued above completes before TMEM is released.
      mma_commit_elect(drain);
      mbar_wait_drain<true>(drain, 0, SITE_TR_DRAIN);
    }
    __syncwarp();
  } else if (warp < 4) {
    regs_dec<C::REGS_CTRL>();
    if constexpr (CODED) {
      // ------------------------------------------------------------------ scales
      // Lane l of the two warps stages tokens t0 and t0 + 64 of each tile, loaded one tile ahead.
      const int t0 = (warp - 2) * 32 + lane;
      int g = 0, qi = 0;
      bool ok = true;
      float ks[2], vs[2];
      auto fetch = [&](const TreePiece& it, int j) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int tok = (it.t0 + j) * 128 + t0 + 64 * x;
          ks[x] = vs[x] = 0.f;
          if (tok < it.len) {
            const int pg = tree_page(p, it.b, tok);
            if (pg >= 0) {
              const long long row = ((long long)pg * p.page_size + tree_page_off(p, tok)) * p.Hkv + it.kvh;
              ks[x] = __ldg(p.k_scale + row);
              vs[x] = __ldg(p.v_scale + row);
            }
          }
        }
      };
      TreeWalk w;
      TreePiece it;
      w.init(p, walk0);
      while (ok && w.next(p, it)) {
        fetch(it, 0);
        if (!(ok = mbar_wait_warp<true>(q_full, qi & 1, SITE_TR_SCALE))) break;
        const float kf = p.scale_log2 * *q_down;
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty);
        for (int j = 0; j < it.n; ++j) {
          const int ss = g % C::NS;
          if (!(ok = mbar_wait_warp<true>(&sc_empty[ss], ((g / C::NS) & 1) ^ 1, SITE_TR_SCALE))) break;
          float* dst = reinterpret_cast<float*>(smem + C::OFF_SC + ss * C::SC_BYTES);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = t0 + 64 * x, tok = (it.t0 + j) * 128 + t;
            // A draft's scale may be anything; the rows that do not see it must not meet it.
            if (tok >= it.len - it.qn && !(fabsf(vs[x]) <= 3.4028234663852886e38f)) {
              vs[x] = 0.f;
              if (tok < it.len) odd_piece[qi & 7] = qi + 1;
            }
            dst[t] = ks[x] * kf;
            dst[128 + t] = vs[x];
            dst[256 + t] = fminf(fmaxf(__log2f(fabsf(vs[x])), C::LOG_MIN), C::LOG_MAX);
          }
          uint32_t k1 = 0, k0 = 0x7f800000u, v1 = 0, v0 = 0x7f800000u;
          bool odd = false;  // K scales that are negative or not finite
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float k = ks[x] * kf;
            odd |= !(k >= 0.f && k <= 3.4028234663852886e38f);
            k1 = max(k1, __float_as_uint(k));
            k0 = min(k0, __float_as_uint(k));
            v1 = max(v1, __float_as_uint(fabsf(vs[x])));
            v0 = min(v0, __float_as_uint(fabsf(vs[x])));
          }
          k1 = __reduce_max_sync(0xffffffffu, k1);
          k0 = __reduce_min_sync(0xffffffffu, k0);
          v1 = __reduce_max_sync(0xffffffffu, v1);
          v0 = __reduce_min_sync(0xffffffffu, v0);
          odd = __any_sync(0xffffffffu, odd);
          if (lane == 0) {
            dst[384 + (warp - 2) * 4] = __uint_as_float(k1);
            dst[385 + (warp - 2) * 4] = odd ? -INFINITY : __uint_as_float(k0);
            dst[386 + (warp - 2) * 4] = fminf(fmaxf(__log2f(__uint_as_float(v1)), C::LOG_MIN), C::LOG_MAX);
            dst[387 + (warp - 2) * 4] = fminf(fmaxf(__log2f(__uint_as_float(v0)), C::LOG_MIN), C::LOG_MAX);
          }
          if (j + 1 < it.n) fetch(it, j + 1);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[ss]);
          ++g;
        }
        ++qi;
      }
    }
  } else if (CODED && warp >= 12) {
    // ------------------------------------------------------------------ converters
    if constexpr (CODED) {
      regs_dec<C::REGS_CONV>();
      const int cw = warp - 12, t = cw * 32 + lane;
      // Lane l of a warp widens 16 codes: row pair 2 (l >> 3) + ((l >> 2) & 1) of eight rows, 16-code column c.  The
      // two rows of a pair take columns 0-3 and 4-7, so the eight lanes of a phase read 128 distinct
      // bytes and their two 16-byte results go to eight distinct chunks of the swizzled tile.
      // One rolled copy of this code serves K and V: unrolled per unit kind it overflowed the instruction
      // cache (4.3 of 17 stall cycles an instruction, 8400 cycles a tile against 1450 of HBM time).
      const int sub = lane & 7, hi_row = sub >> 2;
      const int row0 = cw * 32 + (lane >> 3) * 2 + hi_row;
      int u = 0, qi = 0;
      bool ok = true;
      auto convert = [&](const TreePiece& it, int j, bool is_v) -> bool {
        const int rs = u % C::NR, st = u % C::NU;
        bool r = mbar_wait_warp<true>(&raw_full[rs], (u / C::NR) & 1, SITE_TR_CONV);
        r = r && mbar_wait_warp<true>(&u_empty[st], ((u / C::NU) & 1) ^ 1, SITE_TR_CONV);
        if (!r) return false;
        // Shared addresses: through `smem`, which is aligned by hand, the accesses would be generic ones.
        const uint32_t raw = smem_u32(smem + C::OFF_RAW) + rs * C::RAW_BYTES;
        const uint32_t dst = smem_u32(smem + C::OFF_U) + st * C::TILE_BYTES;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t w4[4][4];
          int col[2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // rows row0 + 16 h + 8 (i >> 1), both halves of their columns
            const int row = row0 + h * 16 + (i >> 1) * 8;
            if (i < 2) col[i] = (sub & 3) + 4 * (hi_row ^ i);
            if constexpr (KIND == TREE_INT4) {
              if (i < 2) col[i] ^= ((lane >> 3) & 1) << 2;  // rows are 64 bytes: the next row pair takes the other half
              const uint2 x = lds_u2(raw + row * 64 + col[i & 1] * 8);
              w4[i][0] = x.x, w4[i][1] = x.y, w4[i][2] = w4[i][3] = 0u;
            } else {
              const uint4 x = lds_u4(raw + row * 128 + col[i & 1] * 16);
              w4[i][0] = x.x, w4[i][1] = x.y, w4[i][2] = x.z, w4[i][3] = x.w;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 lo, hi;
            tree_widen<KIND>(w4[i], lo, hi);
            const int row = row0 + h * 16 + (i >> 1) * 8;
            const uint32_t box = dst + (col[i & 1] >> 2) * C::BOX_BYTES;
            const int ch = (col[i & 1] & 3) * 2;
            sts_u4(box + sw128_offset(row, ch), lo);
            sts_u4(box + sw128_offset(row, ch + 1), hi);
          }
        }
        const int kv0 = (it.t0 + j) * 128, base = it.len - it.qn;
        if (is_v && kv0 + 128 > base) {  // this warp's rows that are drafts, or past them
          const unsigned long long any = tree_seen_any(p, it.b, it.qn, lane);
          const int d = kv0 + t - base;
          __syncwarp();
          if (d >= 0) {
            const bool drop = d >= it.qn || !((any >> d) & 1);
            if (tree_scrub_row<C::NBOX, C::EXP_MASK>(smem + C::OFF_U + st * C::TILE_BYTES, t, drop)) odd_piece[qi & 7] = qi + 1;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&u_full[st]);
          mbar_arrive(&raw_empty[rs]);
        }
        ++u;
        return true;
      };
      // The piece's queries, bf16 -> f16 in place, times a power of two that takes the largest |q| to
      // [2^14, 2^15).  What falls below f16's normal range is then off by at most 2^-39 of the largest.  A row whose
      // own largest is more than 2^14 below that (2^-25 of its own, as little as fp32 accumulation loses on it) is taken
      // there by a power of two of its own, whose ratio to the common one the softmax multiplies its scores by.
      // Thread t holds 16-byte chunk t & 7 of rows t >> 3, + 16, ...: a row belongs to eight lanes of a warp.
      auto q_shift = [](uint32_t top) -> int { return min(14 + 127 - max((int)(top >> 7), 1), 127); };
      auto convert_q = [&](const TreePiece& it) -> bool {
        if (!mbar_wait_warp<true>(q_raw, qi & 1, SITE_TR_CONV)) return false;
        // Only rows of drafts there are: nobody looks at the others, nor at what they turn into.
        const uint32_t qs = smem_u32(smem + C::OFF_Q) + t * 16;
        float* const rowf = row_factor + (qi & 1) * C::NQ * 128;  // first the rows' largest |q|, as bf16 bits
        uint32_t top = 0;
#pragma unroll 1
        for (int s = 0; s < C::NQ; ++s) {
          const int rows = min(max(it.qn - (rb * C::NQ + s) * p.tps, 0), p.tps) * p.G;
#pragma unroll 1
          for (int r0 = 0; r0 + cw * 4 < rows; r0 += 16) {
            const int r = r0 + (t >> 3);
            uint32_t m = 0;
            if (r < rows) {
#pragma unroll
              for (int x = 0; x < C::NBOX; ++x) {
                const uint4 v = lds_u4(qs + s * C::TILE_BYTES + x * C::BOX_BYTES + r0 * 128);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
                  if (lo < 0x7f80u) m = max(m, lo);
                  if (hi < 0x7f80u) m = max(m, hi);
                }
              }
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((lane & 7) == 0 && r < rows) rowf[s * 128 + r] = __uint_as_float(m);
            top = max(top, m);
          }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) {
          q_max[cw] = top;
          mbar_arrive(q_meet);
        }
        // Not a named barrier, whose wait has no limit should another warp have given up.
        if (!mbar_wait_warp<true>(q_meet, qi & 1, SITE_TR_CONV)) return false;
        top = max(max(q_max[0], q_max[1]), max(q_max[2], q_max[3]));
        const int shift = q_shift(top);
        if (t == 0) *q_down = exp2f((float)-shift);
#pragma unroll 1
        for (int s = 0; s < C::NQ; ++s) {
          const int rows = min(max(it.qn - (rb * C::NQ + s) * p.tps, 0), p.tps) * p.G;
#pragma unroll 1
          for (int r0 = 0; r0 + cw * 4 < rows; r0 += 16) {
            const int r = r0 + (t >> 3);
            int row_shift = shift;
            if (r < rows) {
              const uint32_t m = __float_as_uint(rowf[s * 128 + r]);
              if (m > 0 && (m >> 7) + 14 < (top >> 7)) row_shift = q_shift(m);
              const float up = __uint_as_float((uint32_t)(127 + row_shift) << 23);
#pragma unroll
              for (int x = 0; x < C::NBOX; ++x) {
                const uint32_t at = qs + s * C::TILE_BYTES + x * C::BOX_BYTES + r0 * 128;
                const uint4 v = lds_u4(at);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                float f[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  f[2 * k] = __uint_as_float(w[k] << 16) * up;
                  f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * up;
                }
                uint4 h;
                if constexpr (KIND == TREE_INT4)
                  h = make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1], f[5]), pack_f16x2(f[2], f[6]),
                                 pack_f16x2(f[3], f[7]));
                else
                  h = make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                                 pack_f16x2(f[6], f[7]));
                sts_u4(at, h);
              }
            }
            __syncwarp();  // the row's largest has been read
            if ((lane & 7) == 0 && r < rows) rowf[s * 128 + r] = row_shift == shift ? 1.f : exp2f((float)(shift - row_shift));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        return true;
      };
      TreeWalk w;
      TreePiece it;
      w.init(p, walk0);
      while (ok && w.next(p, it)) {
        const int n = it.n;
        const bool duo = paired(it);
        ok = convert_q(it);
        for (int x = 0; x < 2 * n && ok; ++x) {  // the units of the piece, in the order of tree_v_unit
          bool is_v;
          int j;
          if (duo) {
            is_v = x & 1;
            j = x >> 1;
          } else {
            is_v = x == 2 * n - 1 || (x > 0 && !(x & 1));
            j = x == 2 * n - 1 ? n - 1 : is_v ? (x - 2) >> 1 : (x + 1) >> 1;
          }
          ok = convert(it, j, is_v);
        }
        ++qi;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    regs_inc<C::REGS_SOFTMAX>();
    const int slot = (warp - 4) >> 2;
    const int wq = warp & 3;  // TMEM lane quarter this warp may access
    const int r = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + slot * 128 + lane_off;
    const uint32_t tO = tmem + 256 + slot * D + lane_off;
    const int tok_0 = (rb * C::NQ + (PAIR && !C::MIXED ? slot : 0)) * p.tps + r / p.G;
    const int head_g = r % p.G;
    const bool row_used = r < p.tps * p.G && tok_0 < p.n_q;
    int cs = 0, g = 0, qi = 0, ub = 0;  // tiles of this slot, tiles of the CTA, pieces, units before this piece
    bool ok = true;
    // The walk and its piece are kept in shared memory, a copy per warp: between pieces they are dead weight,
    // and the registers they took were spilled scores.
    TreeWalk& sw = reinterpret_cast<TreeWalk*>(smem + C::OFF_WALK)[warp - 4];
    TreePiece& it = reinterpret_cast<TreePiece*>(smem + C::OFF_WALK + 8 * sizeof(TreeWalk))[warp - 4];
    auto next_piece = [&](bool first) -> bool {
      TreeWalk w;
      if (first) w.init(p, walk0);
      else w = sw;
      TreePiece x;
      const bool more = w.next(p, x);
      if constexpr (C::MIXED) x.joins = first ? 0 : it.joins + !paired(it);
      else x.joins = x.idx;
      __syncwarp();  // every lane has read the old walk and piece
      if (lane == 0 && more) {
        sw = w;
        it = x;
      }
      __syncwarp();
      return more;
    };
    while (ok && next_piece(qi == 0)) {
      const int n = it.n, t0 = it.t0, base = it.len - it.qn;
      const bool duo = paired(it);
      const int tok_i = tok_0 + (C::MIXED && duo ? slot * p.tps : 0);  // this row's drafted token
      const bool row_ok = row_used && tok_i < it.qn;
      // This row's mask, read where it is needed (the last tiles of a sequence): no registers in the loop.
      auto row_mask = [&]() -> unsigned long long {
        if (!row_ok) return 0;
        return (unsigned long long)__ldg(p.mask + (long long)it.b * p.n_q + tok_i) & tree_low_bits(it.qn);
      };
      float m_used = -INFINITY, l = 0.f;
      const bool piece_used = __any_sync(0xffffffffu, row_ok);  // else this warp's rows of S, P and O are nobody's
      for (int j = duo ? 0 : slot; j < n; j += duo ? 1 : 2) {
        // tcgen05.ld/st are warp-collective: every lane takes the same branch around them.
        if (!(ok = mbar_wait_warp<true>(&s_full[slot], cs & 1, SITE_TR_SM_S))) break;
        tc_fence_after();
        const int kv0 = (t0 + j) * 128;
        const bool edge = kv0 + 128 > base;
        if (CODED && !piece_used) {  // the tile is only handed on
          if constexpr (CODED) {
            const int ss = (g + j) % C::NS;
            if (!(ok = mbar_wait_warp<true>(&sc_full[ss], ((g + j) / C::NS) & 1, SITE_TR_SM_SC))) break;
            if (lane == 0) mbar_arrive(&sc_empty[ss]);
            if (C::MIXED && !duo && lane == 0) mbar_arrive(&sc_empty[ss]);  // for the other slot's warp too
          }
          if (lane == 0) mbar_arrive(&p_full[slot]);
          ++cs;
          continue;
        }
        // bf16: sr holds the row's 128 scores, read as four chunks of 32.  Coded caches: half of them for the
        // maximum, then two chunks of 16 in turn for the weights; longer loop bodies, of which there are several
        // kinds in flight at once, run out of the instruction cache.
        constexpr int CH = CODED ? 16 : 32;
        uint32_t sr[CODED ? 64 : 128];
        auto chunk = [&](int c) -> uint32_t(&)[CH] {
          return *reinterpret_cast<uint32_t(*)[CH]>(&sr[(CODED ? c & 1 : c) * CH]);
        };
        auto mask_chunk = [&](int c, uint32_t(&x)[CH]) {
          const uint32_t see = tree_seen_word(c * CH, kv0, base, row_mask());
#pragma unroll
          for (int i = 0; i < CH; ++i)
            if (!((see >> i) & 1u)) x[i] = __float_as_uint(-INFINITY);
        };
        uint32_t sc = 0;  // shared address of the tile's scales
        bool rescaled = false;  // coded caches: a row of this warp has a power of two of its own
        const uint32_t row_at = smem_u32(row_factor) + (((qi & 1) * C::NQ + (PAIR && duo ? slot : 0)) * 128 + r) * 4;
        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
        if constexpr (CODED) {
          const int ss = (g + j) % C::NS;
          if (!(ok = mbar_wait_warp<true>(&sc_full[ss], ((g + j) / C::NS) & 1, SITE_TR_SM_SC))) break;
          uint32_t(&h0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
          uint32_t(&h1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[32]);
          sc = smem_u32(smem + C::OFF_SC) + ss * C::SC_BYTES;
          const float rf = row_ok ? lds_f1(row_at) : 1.f;
          bool by_column = edge;
          if (!edge) {
            // The largest bare product times the largest (a negative one: the smallest) K scale, plus the largest
            // log2 |V scale|, bounds the largest sum from above, and from no further than that product times the
            // K scales' range plus the logarithms' range.  A reference within REF_SLACK of the maximum serves;
            // columns are looked at one by one only where it may be farther.
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              tmem_ld32(tS + h * 64, h0);
              tmem_ld32(tS + h * 64 + 32, h1);
              tmem_wait_ld_regs(h0);
              tmem_wait_ld_regs(h1);
#pragma unroll
              for (int i = 0; i < 64; i += 8) {
                mx0 = max3(mx0, __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
                mx1 = max3(mx1, __uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3]));
                mx2 = max3(mx2, __uint_as_float(sr[i + 4]), __uint_as_float(sr[i + 5]));
                mx3 = max3(mx3, __uint_as_float(sr[i + 6]), __uint_as_float(sr[i + 7]));
              }
            }
            const float4 ha = lds_f4(sc + 1536), hb = lds_f4(sc + 1552);
            const float k_max = fmaxf(ha.x, hb.x), k_min = fminf(ha.y, hb.y);
            const float g_max = fmaxf(ha.z, hb.z), g_min = fminf(ha.w, hb.w);
            const float top = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * rf;
            mx0 = fmaf(top, top >= 0.f ? k_max : k_min, g_max);
            mx1 = mx2 = mx3 = -INFINITY;
            // Lanes without a row hold anything, and must not sway which way (and so which rounding) the others take.
            by_column = !__all_sync(0xffffffffu, !row_ok || fmaf(fabsf(top), k_max - k_min, g_max - g_min) <= C::REF_SLACK);
          }
          if (by_column) {
            mx0 = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t(&x)[CH] = chunk(0);
              tmem_ld16(tS + c * CH, x);
              tmem_wait_ld_regs(x);
#pragma unroll
              for (int i = 0; i < CH; i += 4) {
                const float4 k4 = lds_f4(sc + (c * CH + i) * 4), g4 = lds_f4(sc + 1024 + (c * CH + i) * 4);
                const float2 f2 = make_float2(rf, rf);
                const float2 a = fma2(mul2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), f2),
                                      make_float2(k4.x, k4.y), make_float2(g4.x, g4.y));
                const float2 b2 = fma2(mul2(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), f2),
                                       make_float2(k4.z, k4.w), make_float2(g4.z, g4.w));
                x[i] = __float_as_uint(a.x);
                x[i + 1] = __float_as_uint(a.y);
                x[i + 2] = __float_as_uint(b2.x);
                x[i + 3] = __float_as_uint(b2.y);
              }
              if (edge) mask_chunk(c, x);
#pragma unroll
              for (int i = 0; i < CH; i += 4) {
                mx0 = max3(mx0, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                mx1 = max3(mx1, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
              }
            }
          }
          tmem_ld16(tS, chunk(0));  // for the weights
          rescaled = __any_sync(0xffffffffu, rf != 1.f);  // not ahead of the loads of the scores: rf takes its time
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, chunk(c));
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld_regs(chunk(c));
          if (edge) {
#pragma unroll
            for (int c = 0; c < 4; ++c) mask_chunk(c, chunk(c));
          }
#pragma unroll
          for (int i = 0; i < 128; i += 8) {
            mx0 = max3(mx0, __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
            mx1 = max3(mx1, __uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3]));
            mx2 = max3(mx2, __uint_as_float(sr[i + 4]), __uint_as_float(sr[i + 5]));
            mx3 = max3(mx3, __uint_as_float(sr[i + 6]), __uint_as_float(sr[i + 7]));
          }
        }
        // Scores in units of log2: the staged K scales of a coded cache hold the factor already.
        const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
        const float m_tile = CODED ? mx - C::REF_DROP : mx * p.scale_log2;
        const float m_new = fmaxf(m_used, m_tile);
        const bool need = m_new > m_used + C::RESCALE_THRESHOLD;
        if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2_approx(m_used - m_new) : 1.f;  // 0 when m_used = -inf
          if (need) {
            l *= alpha;
            m_used = m_new;
          }
          if (j > (duo ? 0 : slot)) {  // the whole warp rescales its 32 rows of O (factor 1 where unchanged)
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t orow[32];
              tmem_ld32(tO + c * 32, orow);
              tmem_wait_ld_regs(orow);
#pragma unroll
              for (int i = 0; i < 32; ++i) orow[i] = __float_as_uint(__uint_as_float(orow[i]) * alpha);
              tmem_st32(tO + c * 32, orow);
            }
            tmem_wait_st();
          }
        }
        const float neg_m = (m_used == -INFINITY) ? 0.f : -m_used;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 nm2 = make_float2(neg_m, neg_m);
        float2 a0 = make_float2(0.f, 0.f), a1 = a0;  // the row sum, of the unrounded weights
        auto add_sum = [&](int i, float2 e) {
          float2& a = (i & 1) == 0 ? a0 : a1;
          a = add2(a, e);
        };
        if constexpr (CODED) {
          // A masked tile has a copy of its own: selects in the common one cost 1500 cycles a tile.  Rows with a power of two
          // of their own take it too (one head in four 2^20 above the others, b8 n16 t32768 FP8: 198 -> 298 us).
          auto weights = [&](auto masked) {
            const float rf = masked.value ? lds_f1(row_at) : 1.f;
            auto scaled = [&](uint32_t a, uint32_t b) -> float2 {
              const float2 y = make_float2(__uint_as_float(a), __uint_as_float(b));
              return masked.value ? mul2(y, make_float2(rf, rf)) : y;
            };
#pragma unroll 2
            for (int c = 0; c < 8; ++c) {
              uint32_t(&x)[CH] = chunk(c);
              float4 k4[4], v4[4];  // asked for ahead of the waits that come before their use
#pragma unroll
              for (int i = 0; i < 4; ++i) k4[i] = lds_f4(sc + c * 64 + i * 16);
              tmem_wait_ld_regs(x);
              // P lands in columns 8 c .. 8 c + 7, all below the chunk that is still to be read.
              if (c < 7) tmem_ld16(tS + (c + 1) * CH, chunk(c + 1));
#pragma unroll
              for (int i = 0; i < 4; ++i) v4[i] = lds_f4(sc + 512 + c * 64 + i * 16);
#pragma unroll
              for (int i = 0; i < CH; i += 4) {
                const float2 a = fma2(scaled(x[i], x[i + 1]), make_float2(k4[i / 4].x, k4[i / 4].y), nm2);
                const float2 b2 = fma2(scaled(x[i + 2], x[i + 3]), make_float2(k4[i / 4].z, k4[i / 4].w), nm2);
                x[i] = __float_as_uint(a.x);
                x[i + 1] = __float_as_uint(a.y);
                x[i + 2] = __float_as_uint(b2.x);
                x[i + 3] = __float_as_uint(b2.y);
              }
              if (masked.value) mask_chunk(c, x);
              uint32_t pk[8];
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                float2 e0 =
                    make_float2(ex2_approx(__uint_as_float(x[2 * i])), ex2_approx(__uint_as_float(x[2 * i + 1])));
                float2 e1 =
                    make_float2(ex2_approx(__uint_as_float(x[2 * i + 2])), ex2_approx(__uint_as_float(x[2 * i + 3])));
                add_sum(i, e0);
                add_sum(i + 1, e1);
                // The weight times its V scale is rounded once, to f16 (at most 2^-11 of it, or 2^-28 of the row's
                // largest such product: see REF_DROP).
                e0 = mul2(e0, make_float2(v4[i / 2].x, v4[i / 2].y));
                e1 = mul2(e1, make_float2(v4[i / 2].z, v4[i / 2].w));
                pk[i] = pack_f16x2(e0.x, e0.y);
                pk[i + 1] = pack_f16x2(e1.x, e1.y);
              }
              tmem_st8(tS + c * 8, pk);
            }
          };
          if (edge || rescaled) weights(std::true_type{});
          else weights(std::false_type{});
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
            uint32_t(&x)[CH] = chunk(c);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = fma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, nm2);
              const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
              x[2 * i] = __float_as_uint(e.x);
              x[2 * i + 1] = __float_as_uint(e.y);
              // One rounding of the weight to bf16 (at most 2^-8 of it, and the errors of different
              // keys are independent).
              pk[i] = pack_bf16x2(e.x, e.y);
            }
            tmem_st16(tS + c * 16, pk);
          }
        }
        tmem_wait_st();
        if constexpr (!CODED) {
          if (edge && (!PAIR || slot == 0)) {
            // Thread r owns V row r of the tile: zero it if no token sees its slot, and its non-finite
            // elements if some do.
            const int vu = ub + tree_v_unit<PAIR>(j, n), st = vu % C::NU;
            const unsigned long long any = tree_seen_any(p, it.b, it.qn, lane);
            if (!(ok = mbar_wait_warp<true>(&u_full[st], (vu / C::NU) & 1, SITE_TR_SM_V))) break;
            const int d = kv0 + r - base;
            if (d >= 0) {
              const bool drop = d >= it.qn || !((any >> d) & 1);
              if (tree_scrub_row<C::NBOX, C::EXP_MASK>(smem + C::OFF_U + st * C::TILE_BYTES, r, drop)) odd_piece[qi & 7] = qi + 1;
            }
            fence_proxy_async_smem();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&p_full[slot]);
          if constexpr (CODED) {
            mbar_arrive(&sc_empty[(g + j) % C::NS]);
            if (C::MIXED && !duo) mbar_arrive(&sc_empty[(g + j) % C::NS]);
          }
        }
        if constexpr (!CODED) {  // after P is handed over: the MMA does not wait for it
#pragma unroll
          for (int i = 0; i < 64; ++i)
            add_sum(i, make_float2(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1])));
        }
        a0 = add2(a0, a1);
        l += a0.x + a0.y;
        ++cs;
      }
      if (!ok) break;
      // ---- epilogue.  Weights of this slot's and the other half's O (paired: of this slot's alone).
      float f_own, f_other = 0.f, lse2;
      if (duo) {
        f_own = l == 0.f ? 0.f : 1.f / l;
        lse2 = l == 0.f ? -INFINITY : m_used + log2f(l);
      } else {
        float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
        if (it.joins > 0 && !(ok = mbar_wait_warp<true>(ml_empty, (it.joins - 1) & 1, SITE_TR_EPI))) break;
        ml[slot * 128 + r] = make_float2(m_used, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
        if (!(ok = mbar_wait_warp<true>(ml_full, it.joins & 1, SITE_TR_EPI))) break;
        const float2 other = ml[(slot ^ 1) * 128 + r];
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_empty);
        const float m = fmaxf(m_used, other.x);  // a half without a visible key has m = -inf, l = 0
        const float wa = l == 0.f ? 0.f : ex2_approx(m_used - m);
        const float wb = other.y == 0.f ? 0.f : ex2_approx(other.x - m);
        const float sum = l * wa + other.y * wb;
        f_own = sum == 0.f ? 0.f : wa / sum;
        f_other = sum == 0.f ? 0.f : wb / sum;
        lse2 = sum == 0.f ? -INFINITY : m + log2f(sum);
      }
      if (!(ok = mbar_wait_warp<true>(o_full, qi & 1, SITE_TR_EPI))) break;
      tc_fence_after();
      const bool fix = *reinterpret_cast<volatile int*>(odd_piece + (qi & 7)) == qi + 1;
      const long long orow = ((long long)it.b * p.n_q + tok_i) * p.Hq + (long long)it.kvh * p.G + head_g;
      const long long part = (long long)blockIdx.x * 2 + it.which;
      const int prow = (duo ? slot * 128 : 0) + r;
      // Paired: each slot stores its rows' D columns; halves: each slot stores half the columns of every row.
      const int n_ch = duo ? D / 32 : D / 64;
      const int ch0 = duo ? 0 : slot * n_ch;
      if (CODED && !piece_used && lane == 0) mbar_arrive(o_empty);
#pragma unroll 1
      for (int c = ch0; c < ch0 + n_ch && (piece_used || !CODED); ++c) {
        uint32_t ov[32];
        tmem_ld32(tO + c * 32, ov);
        tmem_wait_ld_regs(ov);
#pragma unroll
        for (int i = 0; i < 32; ++i)  // an O that no PV wrote is not read into the sum
          ov[i] = f_own == 0.f ? 0u : __float_as_uint(__uint_as_float(ov[i]) * f_own);
        if (!duo) {
          uint32_t o2[32];
          tmem_ld32(tmem + 256 + (slot ^ 1) * D + lane_off + c * 32, o2);
          tmem_wait_ld_regs(o2);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (f_other != 0.f)
              ov[i] = __float_as_uint(fmaf(__uint_as_float(o2[i]), f_other, __uint_as_float(ov[i])));
        }
        if (c == ch0 + n_ch - 1) {  // O has been read: the next piece's first PV may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty);
        }
        if (row_ok) {
          float out[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) out[i] = __uint_as_float(ov[tree_place<KIND>(i)]);
          if (fix && lse2 != -INFINITY) {
            const unsigned long long m64 = row_mask();  // non-finite values of the drafts this row sees
#pragma unroll 1
            for (int dq = 0; dq < it.qn; ++dq) {
              const int tok = base + dq;
              if (!((m64 >> dq) & 1) || tok < it.t0 * 128 || tok >= (it.t0 + n) * 128) continue;
              const int pg = tree_page(p, it.b, tok);
              if (pg < 0) continue;
              const long long row = ((long long)pg * p.page_size + tree_page_off(p, tok)) * p.Hkv + it.kvh;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float v = tree_v_value<KIND, D>(p, row, c * 32 + i);
                if (!(fabsf(v) <= 3.4028234663852886e38f)) out[i] += v;
              }
            }
          }
          if (it.whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + orow * D + c * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 x;
              x.x = pack_bf16x2(out[8 * i + 0], out[8 * i + 1]);
              x.y = pack_bf16x2(out[8 * i + 2], out[8 * i + 3]);
              x.z = pack_bf16x2(out[8 * i + 4], out[8 * i + 5]);
              x.w = pack_bf16x2(out[8 * i + 6], out[8 * i + 7]);
              dst[i] = x;
            }
          } else {
            // Column by column: 32 rows' neighbouring floats a store (row by row, 16 bytes of 32 rows each, the stores
            // took half of the 12,000 cycles of a piece's epilogue).
            float* dst = p.part_o + (part * D + c * 32) * C::ROWS + prow;
#pragma unroll
            for (int i = 0; i < 32; ++i) dst[i * C::ROWS] = out[i];
          }
        }
      }
      if (row_ok && (duo || slot == 0)) {
        if (!it.whole) p.part_lse[part * C::ROWS + prow] = lse2;
        else if (p.lse) p.lse[orow] = lse2 * 0.69314718055994531f;
      }
      g += n;
      ub += 2 * n;
      ++qi;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the partials of items that several CTAs shared, and writes the rows no tile belongs to.  A block takes 32
// neighbouring rows of a row block (sequence b, KV head) and 8 NC of their columns: a lane per row, NC
// columns per warp, so that partials are read a line at a time.  Rows that one CTA finished are left alone.
template <int D, int NC>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p, int rows_per_part, int slots) {
  __shared__ float weight[kTreeMaxRanges][32];  // of each partial, row by row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = ((int)blockIdx.y * 8 + warp) * NC;
  grid_dependency_wait();
  int x = (int)blockIdx.x;
  const int prow = x % (rows_per_part / 32) * 32 + lane;
  x /= rows_per_part / 32;
  const int rb = x % p.n_rb;
  x /= p.n_rb;
  const int kvh = x % p.Hkv, b = x / p.Hkv;
  const int r = prow & 127, i = (rb * slots + (prow >> 7)) * p.tps + r / p.G;
  const bool used = r < p.tps * p.G && i < p.n_q;
  if (!__any_sync(0xffffffffu, used)) return;
  int total = 0, before = 0;
  for (int y = lane; y < p.B; y += 32) {
    const int n = tree_tiles(p, y);
    total += n;
    if (y < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  const int tiles = tree_tiles(p, b), qn = tree_qlen(p, b);
  const bool wanted = used && i < qn && tiles > 0;
  float acc[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) acc[k] = 0.f;
  float out = -INFINITY;
  if (tiles > 0) {  // the same for the whole block
    const int W = total * p.Hkv, ng = min(p.n_groups, W);
    const int a = before * p.Hkv + kvh * tiles;
    const int g0 = (int)(((long long)(a + 1) * ng - 1) / W), g1 = (int)(((long long)(a + tiles) * ng - 1) / W);
    if (g0 == g1) {  // finished by its CTA
      if (wanted) return;
    } else {
      const int n = g1 - g0 + 1;
      const bool inside = a > tree_range(g0, W, ng);  // the item begins within its first range
      auto part = [&](int k) -> long long {
        return ((long long)(g0 + k) * p.n_rb + rb) * 2 + (k == 0 && inside ? 1 : 0);
      };
      for (int k = warp; k < n; k += 8)
        weight[k][lane] = wanted ? p.part_lse[part(k) * rows_per_part + prow] : -INFINITY;
      __syncthreads();
      float mx = -INFINITY, sum = 0.f;
      bool nan = false;
      for (int k = 0; k < n; ++k) {
        const float y = weight[k][lane];
        nan |= y != y;
        mx = fmaxf(mx, y);
      }
      if (nan) mx = __int_as_float(0x7fc00000);
      if (mx != -INFINITY) {
        const float* src = p.part_o + (long long)c0 * rows_per_part + prow;
#pragma unroll(64 / NC)
        for (int k = 0; k < n; ++k) {
          const float w = ex2_approx(weight[k][lane] - mx);
          sum += w;
          const float* s = src + part(k) * D * rows_per_part;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float y = s[c * rows_per_part];
            acc[c] = w == 0.f ? acc[c] : fmaf(w, y, acc[c]);  // a part that saw nothing holds anything
          }
        }
        out = (mx + log2f(sum)) * 0.69314718055994531f;
        const float inv = 1.f / sum;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[c] *= inv;
      }
    }
  }
  if (!used) return;
  const long long row = ((long long)b * p.n_q + i) * p.Hq + (long long)kvh * p.G + r % p.G;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + c0);
#pragma unroll
  for (int k = 0; k < NC / 2; ++k) dst[k] = pack_bf16x2(acc[2 * k], acc[2 * k + 1]);
  if (p.lse && c0 == 0) p.lse[row] = out;
}

}  // namespace attn
