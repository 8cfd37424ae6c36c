// Keeping a KV cache: the accepted path of a draft tree, and the pages of a paged cache (LLM-CoOpt
// summary, "Opt-Pa": fixed-size pages, mapped on demand; ONNX Runtime packed-QSA analysis, "Code
// analysis" 2: what follows the verification of several tokens).
//
// Nothing here is computed: rows and pages move as bytes, and small integer tables are rewritten on the
// device, so a decoding step never waits for the host.  Cache buffers are K, V and, for coded caches, their
// scales, each [layers, pages, page_size, tok_bytes].
#pragma once

#include "device_ext.cuh"

namespace attn {

struct CacheBufs {
  char* p[4];             // K, V, K scales, V scales
  long long layer[4];     // bytes of a layer
  int tok[4];             // bytes of a token
  int vec[4];             // bytes a thread moves at a time: 16, or 4 (scales whose address or size asks for it)
  int n, n_layers;
  int page_size, num_pages;
};

static constexpr int kCopyThreads = 256;
static constexpr int kCopyCtas = 4;  // a processor, which the kernels' registers have to leave room for: at 72 a thread
                                     // instead of 64 three fit, and a compaction of 4096 pages took 245 us, not 187
static constexpr int kChunkBytes = kCopyThreads * 2 * 16;  // a CTA has two of them in flight
static constexpr int kMaxPages = 1 << 20;                  // bitmaps of pages live in shared memory

// Copies n_items runs of tokens in every layer: item(i, src, dst, n_tok) names the pages and how many tokens.
// What bounds it is HBM.  Segments of up to four 8 KB chunks go round the CTAs of a grid of four per
// processor (one chunk each when there are few); a CTA loads its next chunk before it stores the last.
template <class Item>
__device__ __forceinline__ void copy_items(const CacheBufs& c, long long n_items, Item item) {
  struct Chunk {
    const char* from;
    char* to;
    int bytes;
    bool wide;
  };
  int seg0[5], per = 0;  // first segment of each buffer's page
  long long seg_bytes = kChunkBytes;
#pragma unroll 1
  for (int r = 0; r < 2; ++r) {
    per = 0;
    for (int s = 0; s < c.n; ++s) {
      seg0[s] = per;
      per += (int)(((long long)c.page_size * c.tok[s] + seg_bytes - 1) / seg_bytes);
    }
    if (r > 0 || n_items * c.n_layers * per < 16LL * gridDim.x) break;
    seg_bytes = 4 * kChunkBytes;
  }
  const long long units = n_items * c.n_layers * per;
  long long u = blockIdx.x;
  if (u >= units) return;
  // The CTA's next segments, one found by each thread: what item() costs (a search in the bitmap of live
  // pages, for one) is paid side by side, not in front of every load.
  __shared__ const char* seg_from[kCopyThreads];
  __shared__ char* seg_to[kCopyThreads];
  __shared__ int seg_left[kCopyThreads];  // bytes, negative: moved a word at a time
  int at = 0, known = 0;
  const char* from = nullptr;  // the rest of the current segment
  char* to = nullptr;
  int left = 0;
  bool wide = true;
  auto find = [&](long long v) {
    int seg, s = 0, src, dst, n_tok, layer, i;
    if (units <= 0xffffffffLL) {
      const unsigned r = (unsigned)v / (unsigned)per;
      seg = (int)((unsigned)v - r * (unsigned)per);
      i = (int)(r / (unsigned)c.n_layers);
      layer = (int)(r - (unsigned)i * (unsigned)c.n_layers);
    } else {
      seg = (int)(v % per);
      layer = (int)(v / per % c.n_layers);
      i = (int)(v / per / c.n_layers);
    }
    item(i, src, dst, n_tok);
    while (s + 1 < c.n && seg >= seg0[s + 1]) ++s;
    const long long page = (long long)c.page_size * c.tok[s], off = (seg - seg0[s]) * seg_bytes;
    seg_from[threadIdx.x] = c.p[s] + layer * c.layer[s] + src * page + off;
    seg_to[threadIdx.x] = c.p[s] + layer * c.layer[s] + dst * page + off;
    const int n = src == dst ? 0 : (int)max(0LL, min(seg_bytes, (long long)n_tok * c.tok[s] - off));
    seg_left[threadIdx.x] = c.vec[s] == 16 ? n : -n;
  };
  auto next = [&](Chunk& x) -> bool {
    while (left <= 0) {
      if (at == known) {
        if (u >= units) return false;
        __syncthreads();
        known = (int)min((long long)kCopyThreads, (units - u + gridDim.x - 1) / gridDim.x);
        if ((int)threadIdx.x < known) find(u + (long long)threadIdx.x * gridDim.x);
        u += (long long)known * gridDim.x;
        at = 0;
        __syncthreads();
      }
      from = seg_from[at];
      to = seg_to[at];
      left = abs(seg_left[at]);
      wide = seg_left[at] >= 0;
      ++at;
    }
    x.from = from;
    x.to = to;
    x.bytes = min(left, kChunkBytes);
    x.wide = wide;
    from += kChunkBytes;
    to += kChunkBytes;
    left -= kChunkBytes;
    return true;
  };
  auto load = [&](const Chunk& x, uint4(&v)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int o = (threadIdx.x + i * kCopyThreads) * 16;
      if (x.wide && o < x.bytes) v[i] = *reinterpret_cast<const uint4*>(x.from + o);
    }
  };
  auto store = [&](const Chunk& x, const uint4(&v)[2]) {
    if (x.wide) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int o = (threadIdx.x + i * kCopyThreads) * 16;
        if (o < x.bytes) *reinterpret_cast<uint4*>(x.to + o) = v[i];
      }
    } else {
      for (int o = threadIdx.x * 4; o < x.bytes; o += kCopyThreads * 4)
        *reinterpret_cast<uint32_t*>(x.to + o) = *reinterpret_cast<const uint32_t*>(x.from + o);
    }
  };
  uint4 v[2], w[2];
  Chunk a, b;
  if (!next(a)) return;
  load(a, v);
  while (true) {
    const bool second = next(b);
    if (second) load(b, w);
    store(a, v);
    if (!second) break;
    const bool more = next(a);
    if (more) load(a, v);
    store(b, w);
    if (!more) break;
  }
}

// ------------------------------------------------------------------------------- accepted path

struct AcceptParams {
  CacheBufs c;
  int B, n_q, max_pages;
  const int* page_table;  // or null: sequence b is page b
  const int* kv_lens;
  const int* q_lens;      // or null: n_q
  const int* path;        // [B, n_q]
  const int* n_acc;       // [B]
  int* kv_lens_out;
};

// Block (x, b, layer): columns of tokens, in order of the path.  A thread owns its columns of every moved
// token, so nothing is read after another thread has overwritten it; on a rising path (p_j >= j) rows
// are read in batches ahead of the writes, which only reach slots that later steps do not read.  Any
// other path goes through registers whole, a word at a time.
__global__ void __launch_bounds__(128) tree_accept_kernel(const AcceptParams p) {
  const int b = blockIdx.y, layer = blockIdx.z;
  __shared__ long long from[64], to[64];  // token rows (page * page_size + slot)
  __shared__ int bad, falling;
  const int qn = p.q_lens ? p.q_lens[b] : p.n_q;
  const int len = p.kv_lens[b], acc = p.n_acc[b];
  const int base = len - qn;
  const int cap = p.page_table ? p.max_pages * p.c.page_size : p.c.page_size;
  if (threadIdx.x == 0) {
    bad = qn < 0 || qn > p.n_q || len < 0 || base < 0 || len > cap || acc < 0 || acc > qn;
    falling = 0;
  }
  __syncthreads();
  if (!bad && threadIdx.x < acc) {
    const int j = threadIdx.x, x = p.path[(long long)b * p.n_q + j];
    bool wrong = x < 0 || x >= qn;
    if (!wrong && j > 0 && p.path[(long long)b * p.n_q + j - 1] >= x) falling = 1;
    auto row = [&](int tok) -> long long {
      int pg = b;
      if (p.page_table) {
        pg = p.page_table[(long long)b * p.max_pages + tok / p.c.page_size];
        if (pg < 0 || pg >= p.c.num_pages) wrong = true;
        tok %= p.c.page_size;
      }
      return (long long)pg * p.c.page_size + tok;
    };
    if (!wrong) {
      to[j] = row(base + j);
      from[j] = row(base + x);
    }
    if (wrong) bad = 1;
  }
  __syncthreads();
  if (bad) {  // left as it was
    if (threadIdx.x == 0 && blockIdx.x == 0 && layer == 0) {
      p.kv_lens_out[b] = len;
      record_arg_error(ATTN_DEV_BAD_INDEX, SITE_ACCEPT);
    }
    return;
  }
  if (threadIdx.x == 0 && blockIdx.x == 0 && layer == 0) p.kv_lens_out[b] = base + acc;
  int col = blockIdx.x * 128 + threadIdx.x, s = 0;
  for (; s < p.c.n; ++s) {
    const int cols = p.c.tok[s] / p.c.vec[s];
    if (col < cols) break;
    col -= cols;
  }
  if (s == p.c.n) return;
  const int tok = p.c.tok[s], vec = p.c.vec[s];
  char* mem = p.c.p[s] + layer * p.c.layer[s] + col * vec;
  if (falling) {
    for (int w = 0; w < vec; w += 4) {
      uint32_t x[64];
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (j < acc) x[j] = *reinterpret_cast<const uint32_t*>(mem + from[j] * tok + w);
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (j < acc) *reinterpret_cast<uint32_t*>(mem + to[j] * tok + w) = x[j];
    }
  } else if (vec == 16) {
    for (int j0 = 0; j0 < acc; j0 += 8) {
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j0 + i < acc && from[j0 + i] != to[j0 + i])
          x[i] = *reinterpret_cast<const uint4*>(mem + from[j0 + i] * tok);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j0 + i < acc && from[j0 + i] != to[j0 + i]) *reinterpret_cast<uint4*>(mem + to[j0 + i] * tok) = x[i];
    }
  } else {
    for (int j = 0; j < acc; ++j)
      if (from[j] != to[j])
        *reinterpret_cast<uint32_t*>(mem + to[j] * tok) = *reinterpret_cast<const uint32_t*>(mem + from[j] * tok);
  }
}

// ------------------------------------------------------------------------------- page copies

struct CopyParams {
  CacheBufs c;
  const int* src;
  const int* dst;
  int n;
};

// Every CTA checks the whole list itself (a bitmap of destinations, n reads from L2), so that all of them
// refuse a list whose pages are out of range, written twice, or both written and read.
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) pages_copy_kernel(const CopyParams p) {
  extern __shared__ uint32_t written[];
  __shared__ int bad;
  const int words = (p.c.num_pages + 31) / 32;
  for (int i = threadIdx.x; i < words; i += kCopyThreads) written[i] = 0;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kCopyThreads) {
    const int a = p.src[i], d = p.dst[i];
    if (a < 0 || a >= p.c.num_pages || d < 0 || d >= p.c.num_pages) bad = 1;
    else if (a != d && (atomicOr(&written[d >> 5], 1u << (d & 31)) >> (d & 31)) & 1u) bad = 1;
  }
  __syncthreads();
  if (!bad)
    for (int i = threadIdx.x; i < p.n; i += kCopyThreads) {
      const int a = p.src[i];
      if (a != p.dst[i] && (written[a >> 5] >> (a & 31)) & 1u) bad = 1;
    }
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_arg_error(ATTN_DEV_BAD_INDEX, SITE_PAGES_COPY);
    return;
  }
  copy_items(p.c, p.n, [&](int i, int& src, int& dst, int& n_tok) {
    src = p.src[i];
    dst = p.dst[i];
    n_tok = p.c.page_size;
  });
}

// ------------------------------------------------------------------------------- compaction

struct CompactParams {
  CacheBufs c;
  const int* table;
  long long n_entries;  // B * max_pages
  const int* refs;
  int* table_out;
  int* refs_out;
  int* page_map;
  int* info;  // live pages, moved pages
};

// Pages that are live, as a bitmap with the number of live pages before each group of 128.
struct LivePages {
  const uint4* bits;
  const int* before;
  int groups;
  __device__ __forceinline__ static uint32_t word(const uint4& g, int i) {
    return i == 0 ? g.x : i == 1 ? g.y : i == 2 ? g.z : g.w;
  }
  __device__ __forceinline__ bool live(int p) const { return (word(bits[p >> 7], (p >> 5) & 3) >> (p & 31)) & 1u; }
  __device__ __forceinline__ int rank(int p) const {  // live pages below p
    const uint4 g = bits[p >> 7];
    int r = before[p >> 7];
    const int w = (p >> 5) & 3;
    if (w > 0) r += __popc(g.x);
    if (w > 1) r += __popc(g.y);
    if (w > 2) r += __popc(g.z);
    return r + __popc(word(g, w) & ((1u << (p & 31)) - 1u));
  }
  // The k-th page (from 0) that is live (or, free), given that there is one.
  __device__ __forceinline__ int select(int k, bool free_pages) const {
    int lo = 0, hi = groups - 1;  // the last group with at most k such pages before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      const int n = free_pages ? mid * 128 - before[mid] : before[mid];
      if (n <= k) lo = mid;
      else hi = mid - 1;
    }
    k -= free_pages ? lo * 128 - before[lo] : before[lo];
    const uint4 g = bits[lo];
    int p = lo * 128;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = free_pages ? ~word(g, w) : word(g, w);
      const int n = __popc(x);
      if (k >= n) {
        k -= n;
        p += 32;
        continue;
      }
      uint32_t y = x;
      for (int i = 0; i < k; ++i) y &= y - 1;
      return p + __ffs(y) - 1;
    }
    return p;
  }
};

// Live pages at or past n_live move into the free ones below, both in rising order.  Every CTA builds the
// bitmap and its prefix itself (4 bytes a page from L2): one launch, and no CTA waits for another.
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) pages_compact_kernel(const CompactParams p) {
  extern __shared__ uint4 bits[];
  __shared__ int warp_sum[kCopyThreads / 32];
  const int N = p.c.num_pages, groups = (N + 127) / 128;
  int* before = reinterpret_cast<int*>(bits + groups);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool negative = false;
  // A thread takes whole words: the loads are 16 bytes, eight in flight.
  for (int w = threadIdx.x; w < groups * 4; w += kCopyThreads) {
    uint32_t x = 0;
    const int p0 = w * 32;
    if (p0 + 32 <= N && (reinterpret_cast<uintptr_t>(p.refs) & 15) == 0) {
      int4 r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = reinterpret_cast<const int4*>(p.refs + p0)[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x |= (uint32_t)(r[i].x > 0) << (4 * i) | (uint32_t)(r[i].y > 0) << (4 * i + 1) |
             (uint32_t)(r[i].z > 0) << (4 * i + 2) | (uint32_t)(r[i].w > 0) << (4 * i + 3);
        negative |= (r[i].x | r[i].y | r[i].z | r[i].w) < 0;
      }
    } else {
      for (int i = 0; i < 32 && p0 + i < N; ++i) {
        const int r = p.refs[p0 + i];
        x |= (uint32_t)(r > 0) << i;
        negative |= r < 0;
      }
    }
    reinterpret_cast<uint32_t*>(bits)[w] = x;
  }
  // A count below zero says nothing about who holds the page: whatever moved could land on somebody's.  Every CTA has
  // read every count, so all of them leave here together, with the old numbers as the new ones.
  if (__syncthreads_or(negative)) {
    const long long stride = (long long)gridDim.x * kCopyThreads, first = (long long)blockIdx.x * kCopyThreads + threadIdx.x;
    for (long long i = first; i < N; i += stride) {
      p.page_map[i] = (int)i;
      p.refs_out[i] = p.refs[i];
    }
    for (long long i = first; i < p.n_entries; i += stride) p.table_out[i] = p.table[i];
    if (first == 0) {
      p.info[0] = -1;
      p.info[1] = 0;
      record_arg_error(ATTN_DEV_BAD_INDEX, SITE_PAGES_COMPACT);
    }
    return;
  }
  int total = 0;
  for (int g0 = 0; g0 < groups; g0 += kCopyThreads) {
    const int g = g0 + threadIdx.x;
    int n = 0;
    if (g < groups) {
      const uint4 x = bits[g];
      n = __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w);
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int prior = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kCopyThreads / 32; ++i) {
      if (i < warp) prior += warp_sum[i];
      all += warp_sum[i];
    }
    if (g < groups) before[g] = total + prior + incl - n;
    total += all;
    __syncthreads();
  }
  const int n_live = total;
  const LivePages L{bits, before, groups};
  const int low = n_live < N ? L.rank(n_live) : n_live;  // live pages that stay
  const int moved = n_live - low;
  const long long stride = (long long)gridDim.x * kCopyThreads, first = (long long)blockIdx.x * kCopyThreads + threadIdx.x;
  auto place = [&](int page) {  // where a page goes, -1 for a free one
    if (!L.live(page)) return -1;
    return page < n_live ? page : L.select(L.rank(page) - low, true);
  };
  for (long long i = first; i < N; i += stride) {
    const int page = (int)i;
    p.page_map[page] = place(page);
    int r = 0;
    if (page < n_live) r = L.live(page) ? p.refs[page] : p.refs[L.select(low + page - L.rank(page), false)];
    p.refs_out[page] = r;
  }
  bool wrong = false;
  for (long long i = first; i < p.n_entries; i += stride) {
    const int t = p.table[i];
    wrong |= t >= N;
    p.table_out[i] = t < 0 || t >= N ? -1 : place(t);
  }
  if (wrong) record_arg_error(ATTN_DEV_BAD_INDEX, SITE_PAGES_COMPACT);
  if (first == 0) {
    p.info[0] = n_live;
    p.info[1] = moved;
  }
  copy_items(p.c, moved, [&](int k, int& src, int& dst, int& n_tok) {
    src = L.select(low + k, false);
    dst = L.select(k, true);
    n_tok = p.c.page_size;
  });
}

// ------------------------------------------------------------------------------- fork

struct ForkParams {
  CacheBufs c;
  int B, n_child, max_pages;
  const int* table;
  const int* lens;
  const int* refs;
  const int* parents;
  const int* keep;
  const int* new_lens;
  int* table_out;
  int* lens_out;
  int* refs_out;
  int* info;     // free pages left (or short of, below zero), status
  // workspace
  int* child;    // [n_child] start * 2 + own: its first fresh page in `fresh`, and whether it keeps the page it cuts
  int* copies;   // [n_child][3] source, destination, tokens
  int* fresh;    // [num_pages] free pages in rising order, as many as are taken
  int* count;    // refs after, when they do not fit in shared memory
  int* claim;
  int* head;     // {copies, failed}
};

static constexpr int kForkThreads = 1024;

// What a child keeps of its parent: tokens clamped as documented, whole pages, and whether it cuts a page.
struct ForkKeep {
  int parent, keep, full, held;
  bool cut;
};
__device__ __forceinline__ ForkKeep fork_keep(const ForkParams& p, int c) {
  ForkKeep k;
  k.parent = p.parents[c];
  const int old = k.parent >= 0 ? p.lens[k.parent] : 0, want = p.new_lens[c];
  k.keep = max(0, min(min(p.keep[c], old), want));
  k.full = k.keep / p.c.page_size;
  k.cut = k.keep % p.c.page_size > 0;
  k.held = (int)(((long long)want + p.c.page_size - 1) / p.c.page_size);
  return k;
}

// Exclusive sum over the block of one value per thread; *total gets the block's sum.
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int w = scratch[lane];
    int x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    scratch[lane] = x - w;
    if (lane == 31) scratch[32] = x;
  }
  __syncthreads();
  *total = scratch[32];
  const int r = scratch[warp] + incl - v;
  __syncthreads();
  return r;
}

// The tables, in one CTA (the steps depend on one another through every page's count).  SMEM: counts and
// claims in shared memory, else in the workspace.
template <bool SMEM>
__global__ void __launch_bounds__(kForkThreads) pages_fork_plan_kernel(const ForkParams p) {
  extern __shared__ int fork_smem[];
  __shared__ int scratch[33];
  __shared__ int bad, n_copies;
  const int N = p.c.num_pages, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int page = p.c.page_size;
  grid_launch_dependents();  // pages_fork_apply_kernel's CTAs wait on the other processors
  int* cnt = SMEM ? fork_smem : p.count;
  int* claim = SMEM ? fork_smem + N : p.claim;
  if (tid == 0) bad = n_copies = 0;
  bool wrong = false;
  for (int i = tid; i < N; i += kForkThreads) {
    const int r = p.refs[i];
    wrong |= r < 0;
    cnt[i] = r;
    claim[i] = 0x7fffffff;
  }
  __syncthreads();
  // 1. Lengths and parents, before anything is indexed by them.
  const long long cap = (long long)p.max_pages * page;
  for (int b = tid; b < p.B; b += kForkThreads) wrong |= p.lens[b] < 0 || p.lens[b] > cap;
  for (int c = tid; c < p.n_child; c += kForkThreads) {
    const int a = p.parents[c];
    wrong |= a < -1 || a >= p.B || p.new_lens[c] < 0 || p.new_lens[c] > cap;
  }
  if (wrong) bad = 1;
  __syncthreads();
  // 2. Every old reference goes (a warp per sequence; a count that is used up is a wrong one), then whole kept
  // pages are referenced again.
  if (!bad)
    for (int b = warp; b < p.B; b += kForkThreads / 32) {
      const int held = (int)(((long long)p.lens[b] + page - 1) / page);
      for (int i = lane; i < held; i += 32) {
        const int t = p.table[(long long)b * p.max_pages + i];
        if (t < 0 || t >= N || atomicSub(&cnt[t], 1) < 1) wrong = true;
      }
    }
  __syncthreads();  // nobody reads `bad` any more
  if (wrong) bad = 1;
  __syncthreads();
  if (!bad)
    for (int c = warp; c < p.n_child; c += kForkThreads / 32) {
      const ForkKeep k = fork_keep(p, c);
      for (int i = lane; i < k.full; i += 32) atomicAdd(&cnt[p.table[(long long)k.parent * p.max_pages + i]], 1);
    }
  __syncthreads();
  // 3. A cut page nobody else holds goes to the first child that cuts it.
  if (!bad)
    for (int c = tid; c < p.n_child; c += kForkThreads) {
      const ForkKeep k = fork_keep(p, c);
      if (!k.cut) continue;
      const int x = p.table[(long long)k.parent * p.max_pages + k.full];
      if (cnt[x] == 0) atomicMin(&claim[x], c);
    }
  __syncthreads();
  // 4. Pages each child needs, and where its run of fresh pages starts.
  int total = 0;
  if (!bad)
    for (int c0 = 0; c0 < p.n_child; c0 += kForkThreads) {
      const int c = c0 + tid;
      int need = 0, own = 0;
      if (c < p.n_child) {
        const ForkKeep k = fork_keep(p, c);
        if (k.cut) own = claim[p.table[(long long)k.parent * p.max_pages + k.full]] == c;
        need = k.held - k.full - own;
      }
      int sum;
      const int start = total + block_scan(need, scratch, &sum);
      if (c < p.n_child) p.child[c] = start * 2 + own;  // start < 2^30: checked on the host
      total += sum;
    }
  __syncthreads();
  // 5. Owned pages count, then the free ones are listed (a warp per run of pages).
  const int run = (N + 32 * 32 - 1) / (32 * 32) * 32;
  const int r0 = min(warp * run, N), r1 = min(r0 + run, N);
  int n = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    if (!bad && claim[i] != 0x7fffffff) cnt[i] = 1;
    n += cnt[i] == 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  int n_free;
  int rank = block_scan(lane == 0 ? n : 0, scratch, &n_free);
  rank = __shfl_sync(0xffffffffu, rank, 0);
  const bool fail = bad || n_free < total;
  if (!fail) {
    for (int i0 = r0; i0 < r1 && rank < total; i0 += 32) {
      const int i = i0 + lane;
      const bool is_free = i < r1 && cnt[i] == 0;
      const uint32_t m = __ballot_sync(0xffffffffu, is_free);
      const int at = rank + __popc(m & ((1u << lane) - 1u));
      if (is_free && at < total) {
        p.fresh[at] = i;
        cnt[i] = 1;
      }
      rank += __popc(m);
    }
  }
  __syncthreads();
  for (int i = tid; i < N; i += kForkThreads) p.refs_out[i] = fail ? p.refs[i] : cnt[i];
  // 6. Cut pages that are copied.
  for (int c = tid; c < p.n_child; c += kForkThreads) {
    p.lens_out[c] = fail ? 0 : p.new_lens[c];
    if (fail) continue;
    const ForkKeep k = fork_keep(p, c);
    const int x = p.child[c];
    if (k.cut && !(x & 1)) {
      const int at = atomicAdd(&n_copies, 1);
      p.copies[at * 3] = p.table[(long long)k.parent * p.max_pages + k.full];
      p.copies[at * 3 + 1] = p.fresh[x >> 1];
      p.copies[at * 3 + 2] = k.keep % page;
    }
  }
  __syncthreads();
  if (tid == 0) {
    p.info[0] = bad ? 0 : n_free - total;
    p.info[1] = bad ? 1 : (fail ? 4 : 0);  // ATTN_ERR_INVALID_ARG, ATTN_ERR_BUDGET
    p.head[0] = n_copies;
    p.head[1] = fail;
    if (bad) record_arg_error(ATTN_DEV_BAD_INDEX, SITE_PAGES_FORK);
  }
}

// The new table's rows and the kept parts of cut pages, over the whole GPU.
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) pages_fork_apply_kernel(const ForkParams p) {
  grid_dependency_wait();
  const bool fail = p.head[1];
  const int n_copies = p.head[0];
  const long long entries = (long long)p.n_child * p.max_pages;
  for (long long i = (long long)blockIdx.x * kCopyThreads + threadIdx.x; i < entries;
       i += (long long)gridDim.x * kCopyThreads) {
    const int c = (int)(i / p.max_pages), j = (int)(i % p.max_pages);
    int t = -1;
    if (!fail) {
      const ForkKeep k = fork_keep(p, c);
      const int x = p.child[c], own = x & 1;
      if (j < k.full + own) t = p.table[(long long)k.parent * p.max_pages + j];
      else if (j < k.held) t = p.fresh[(x >> 1) + j - k.full - own];
    }
    p.table_out[i] = t;
  }
  copy_items(p.c, n_copies, [&](int i, int& src, int& dst, int& n_tok) {
    src = p.copies[i * 3];
    dst = p.copies[i * 3 + 1];
    n_tok = p.copies[i * 3 + 2];
  });
}

}  // namespace attn
