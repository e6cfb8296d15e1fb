// Slot embeddings and the gradient of the embedding table.
//
// "DFlash Draft Body", How It Works step 2: the caller supplies an embedding per block
// position -- the anchor token's at slot 0, the mask token's at the others.  The forward is
// a scaled row gather.  The gradient of the table is, for every token, the sum of the slot
// gradients that carry it.  A drafted batch has one very long run (the mask token holds
// gamma of every gamma + 1 slots) and many runs of one, so the slots are sorted by token
// (stably: sums have one fixed order) and the sorted list is cut into equal chunks whatever
// the runs: a CTA sums its chunk run by run, writes the runs that lie inside it, and leaves
// the one or two that cross its ends as fp32 partial rows that a second pass joins in order.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace dflash {

namespace {

constexpr int kThreads = 256;

// ---- forward -------------------------------------------------------------------------

// kN consecutive elements (one, or 16 aligned bytes) as loaded, and as floats
template <typename T, int kN>
struct Raw {
  uint4 u;
};
template <typename T>
struct Raw<T, 1> {
  T u;
};
template <typename T, int kN>
__device__ __forceinline__ Raw<T, kN> load_raw(const T* p) {
  Raw<T, kN> r;
  if constexpr (kN == 1) r.u = __ldg(p);
  else r.u = __ldg(reinterpret_cast<const uint4*>(p));
  return r;
}
template <typename T, int kN>
__device__ __forceinline__ void expand(const Raw<T, kN>& r, float* v) {
  if constexpr (kN == 1) {
    v[0] = to_f(r.u);
  } else {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(w[e]);
    }
  }
}
template <typename T, int kN>
__device__ __forceinline__ void load_pack(const T* p, float* v) {
  expand<T, kN>(load_raw<T, kN>(p), v);
}

// kN consecutive elements, rounded to nearest; the address is aligned to kN elements
template <typename T, int kN>
__device__ __forceinline__ void store_pack(T* p, const float* v) {
  if constexpr (kN == 1) {
    *p = from_f<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < kN; e += 4)
      __stcs(reinterpret_cast<float4*>(p + e), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
  } else {
    uint32_t w[kN / 2];
#pragma unroll
    for (int e = 0; e < kN / 2; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (kN == 8)
      __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
  }
}

// A CTA writes `rows` consecutive slots: tx threads across a row, each with up to kHold packs
// of it in registers, kThreads / tx rows of slots side by side.  A slot with the token of the
// slot before it (the mask token's slots of a block) is stored from the registers; four
// slots' loads are in flight at a time.  Bound by the writes: 8192 x 4096 bf16 slots of 512
// anchors 13.0 us (5.2 TB/s; one slot per CTA read the mask token's row from L2 every time,
// 17.1 us).
constexpr int kHold = 2, kBatch = 4, kMaxRows = 64;

template <typename T, int kN>
__global__ void __launch_bounds__(kThreads)
embed_kernel(const T* __restrict__ table, int V, int D, const int32_t* __restrict__ ids, int Tn,
             float scale, T* __restrict__ out, int tx, int rows, unsigned* status) {
  pdl_wait();
  pdl_trigger();
  __shared__ int s_id[kMaxRows];
  const int x = threadIdx.x & (tx - 1), y = threadIdx.x / tx, ny = kThreads / tx;
  const int t0 = blockIdx.x * rows, n = min(rows, Tn - t0);
  const int nvec = D / kN;
  if ((int)threadIdx.x < n) {
    int id = ids[t0 + threadIdx.x];
    if (id < 0 || id >= V) {
      if (id != -1 && blockIdx.y == 0) report(status, kStatusCheck, kKernEmbed);
      id = -1;
    }
    s_id[threadIdx.x] = id;
  }
  __syncthreads();
  const int c0 = blockIdx.y * (kHold * tx) + x;
  const int share = (n + ny - 1) / ny;  // consecutive slots of one y
  const int r1 = min(n, (y + 1) * share);
  float v[kBatch][kHold][kN];
  int last = -2;                        // the token in v[kBatch - 1]
  for (int r0 = y * share; r0 < r1; r0 += kBatch) {
    int id[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) id[q] = r0 + q < r1 ? s_id[r0 + q] : -2;
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int before = q ? id[q - 1] : last;
      if (id[q] >= 0 && id[q] != before) {
#pragma unroll
        for (int h = 0; h < kHold; ++h)
          if (c0 + h * tx < nvec)
            load_pack<T, kN>(table + (size_t)id[q] * D + (size_t)(c0 + h * tx) * kN, v[q][h]);
      } else if (q == 0) {
        // the row of the batch before goes on: out of the last slot's registers before that
        // slot's own load (scaled already)
#pragma unroll
        for (int h = 0; h < kHold; ++h)
#pragma unroll
          for (int e = 0; e < kN; ++e) v[0][h][e] = v[kBatch - 1][h][e];
      }
    }
    const int was = last;
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const bool same = id[q] == (q ? id[q - 1] : was);
      if (id[q] == -2) break;
#pragma unroll
      for (int h = 0; h < kHold; ++h) {
#pragma unroll
        for (int e = 0; e < kN; ++e)
          v[q][h][e] = id[q] < 0 ? 0.f : same ? v[q ? q - 1 : 0][h][e] : v[q][h][e] * scale;
        if (c0 + h * tx < nvec)
          store_pack<T, kN>(out + (size_t)(t0 + r0 + q) * D + (size_t)(c0 + h * tx) * kN, v[q][h]);
      }
    }
    last = id[kBatch - 1];
  }
}

// ---- sorting the slots by token ------------------------------------------------------
// Keys: the token, or V for slots without one (they sort to the end and are never summed).

__device__ __forceinline__ int slot_key(const int32_t* ids, int t, int V, unsigned* status,
                                        bool tell) {
  const int id = ids[t];
  if (id >= 0 && id < V) return id;
  if (tell && id != -1) report(status, kStatusCheck, kKernEmbed);
  return V;
}

// The table's zeros, written by the CTAs of the first sorting kernel behind its own `ctas`: rows
// that slots carry are written again by the sums.  151936 x 4096 fp32: 2.49 GB at 7.1 TB/s;
// leaving those rows out needs the sorted tokens first and a look-up per row, and was slower
// (420 against 377 us for the whole gradient of 8192 slots).
struct Fill {
  void* p;
  size_t bytes;
};

__device__ __forceinline__ void fill_zero(const Fill& f, unsigned cta, unsigned ctas) {
  float4* p = static_cast<float4*>(f.p);
  const size_t n = f.bytes / 16, step = (size_t)ctas * blockDim.x;
  for (size_t i = (size_t)cta * blockDim.x + threadIdx.x; i < n; i += step)
    p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (cta == 0 && threadIdx.x < f.bytes % 16 / 2)
    reinterpret_cast<uint16_t*>(p + n)[threadIdx.x] = 0;
}

// Up to kRankMax slots: each slot's place is the number of slots before it, counted.  A CTA
// places 64 slots; a warp holds 32 of them and counts one eighth of each tile of keys, which
// all its lanes read from the same shared-memory words.  Quadratic: added to a 64-wide table,
// 512 slots take 13 us (24 us by radix passes), 8192 take 33 (33), 16384 take 74 (40).
constexpr int kRankMax = 8192;
constexpr int kRankTile = 2048;

__global__ void __launch_bounds__(512)
rank_kernel(const int32_t* __restrict__ ids, int Tn, int V, int32_t* __restrict__ key_out,
            int32_t* __restrict__ slot_out, unsigned ctas, Fill fill, unsigned* status) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= ctas) {
    fill_zero(fill, blockIdx.x - ctas, gridDim.x - ctas);
    return;
  }
  __shared__ __align__(16) int keys[kRankTile];
  __shared__ int cnt[64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp & 1, part = warp >> 1;      // 2 groups of 32 slots, 8 parts
  const int t0 = blockIdx.x * 64 + group * 32, t = t0 + lane;
  if (threadIdx.x < 64) cnt[threadIdx.x] = 0;
  const int mine = t < Tn ? slot_key(ids, t, V, status, part == 0) : 0x7fffffff;
  int n = 0;
  for (int base = 0; base < Tn; base += kRankTile) {
    __syncthreads();
    const int each = min(kRankTile, (Tn - base + 31) / 32 * 32) / 8;  // keys per part
    for (int i = threadIdx.x; i < each * 8; i += 512)
      keys[i] = base + i < Tn ? slot_key(ids, base + i, V, status, false) : 0x7fffffff;
    __syncthreads();
    const int p0 = part * each;
#pragma unroll 4
    for (int i = p0; i < p0 + each; i += 4) {
      const int4 k = *reinterpret_cast<const int4*>(keys + i);
      const int s = base + i;                        // 4 slots, all before, in, or behind the group
      if (s + 4 <= t0) {
        n += (k.x <= mine) + (k.y <= mine) + (k.z <= mine) + (k.w <= mine);
      } else if (s >= t0 + 32) {
        n += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
      } else {
        n += (k.x < mine || (k.x == mine && s < t)) + (k.y < mine || (k.y == mine && s + 1 < t)) +
             (k.z < mine || (k.z == mine && s + 2 < t)) +
             (k.w < mine || (k.w == mine && s + 3 < t));
      }
    }
  }
  if (t < Tn) atomicAdd(&cnt[group * 32 + lane], n);
  __syncthreads();
  if (part == 0 && t < Tn) {
    const int at = cnt[group * 32 + lane];
    key_out[at] = mine;
    slot_out[at] = t;
  }
}

// More slots: least-significant-digit radix passes of 9 bits -- per-tile counts, one scan
// over (digit, tile), a stable scatter.
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kTile = 2048;  // slots per CTA: 8 warps of 8 rounds of 32

__device__ __forceinline__ int radix_key(const int32_t* keys, const int32_t* ids, int i, int V,
                                         unsigned* status, bool tell) {
  return keys ? keys[i] : slot_key(ids, i, V, status, tell);
}

__global__ void __launch_bounds__(kThreads)
radix_count_kernel(const int32_t* __restrict__ keys, const int32_t* __restrict__ ids, int Tn,
                   int V, int shift, int tiles, uint32_t* __restrict__ hist, Fill fill,
                   unsigned* status) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= tiles) {
    fill_zero(fill, blockIdx.x - tiles, gridDim.x - tiles);
    return;
  }
  __shared__ uint32_t h[kDigits];
  for (int i = threadIdx.x; i < kDigits; i += kThreads) h[i] = 0;
  __syncthreads();
  const int base = blockIdx.x * kTile;
  for (int i = threadIdx.x; i < kTile; i += kThreads)
    if (base + i < Tn)
      atomicAdd(&h[radix_key(keys, ids, base + i, V, status, true) >> shift & (kDigits - 1)], 1u);
  __syncthreads();
  for (int i = threadIdx.x; i < kDigits; i += kThreads) hist[(size_t)i * tiles + blockIdx.x] = h[i];
}

__global__ void __launch_bounds__(1024)
radix_scan_kernel(uint32_t* __restrict__ hist, int n) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t ws[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t carry = 0;
  for (int base = 0; base < n; base += 4096) {
    uint32_t v[4];
    uint32_t s = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = base + threadIdx.x * 4 + e;
      v[e] = i < n ? hist[i] : 0;
      s += v[e];
    }
    uint32_t incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) ws[warp] = incl;
    __syncthreads();
    uint32_t before = carry, total = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += ws[w];
      total += ws[w];
    }
    carry += total;
    uint32_t at = before + incl - s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = base + threadIdx.x * 4 + e;
      if (i < n) hist[i] = at;
      at += v[e];
    }
  }
}

__global__ void __launch_bounds__(kThreads)
radix_scatter_kernel(const int32_t* __restrict__ keys, const int32_t* __restrict__ slots,
                     const int32_t* __restrict__ ids, int Tn, int V, int shift, int tiles,
                     const uint32_t* __restrict__ offs, int32_t* __restrict__ key_out,
                     int32_t* __restrict__ slot_out, unsigned* status) {
  pdl_wait();
  pdl_trigger();
  constexpr int kWarps = kThreads / 32, kRounds = kTile / kThreads;
  __shared__ uint32_t wh[kWarps][kDigits];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kWarps * kDigits; i += kThreads) (&wh[0][0])[i] = 0;
  __syncthreads();
  const int base = blockIdx.x * kTile + warp * (kTile / kWarps);
  int key[kRounds], slot[kRounds];
  uint32_t rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int i = base + r * 32 + lane;
    const bool in = i < Tn;
    key[r] = in ? radix_key(keys, ids, i, V, status, false) : 0;
    slot[r] = in ? (slots ? slots[i] : i) : 0;
    const int d = in ? key[r] >> shift & (kDigits - 1) : kDigits;
    const unsigned peers = __match_any_sync(0xffffffffu, d);
    const uint32_t before = in ? wh[warp][d] : 0;
    rank[r] = before + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (in && lane == __ffs(peers) - 1) wh[warp][d] = before + __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kThreads) {
    uint32_t at = offs[(size_t)d * tiles + blockIdx.x];
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t n = wh[w][d];
      wh[w][d] = at;
      at += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (base + r * 32 + lane < Tn) {
      const uint32_t at = wh[warp][key[r] >> shift & (kDigits - 1)] + rank[r];
      key_out[at] = key[r];
      slot_out[at] = slot[r];
    }
  }
}

// ---- sums over the sorted slots --------------------------------------------------------

struct GradArgs {
  const void* grad;
  const int32_t* key;    // [T] sorted, V for slots without a token
  const int32_t* slot;   // [T]
  int T, V, D;
  float scale;
  int accumulate;
  void* table;
  float* part;           // [2 * chunks][D]: a chunk's head (even) and tail (odd) partial rows
  int chunk, chunks, col_tiles;
};

template <typename TT, int kN>
__device__ __forceinline__ void write_row(const GradArgs& a, int v, int col, const float* s) {
  TT* p = static_cast<TT*>(a.table) + (size_t)v * a.D + col;
  float r[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) r[e] = s[e] * a.scale;
  if (a.accumulate) {
#pragma unroll
    for (int e = 0; e < kN; ++e) r[e] += to_f(p[e]);
  }
  store_pack<TT, kN>(p, r);
}

template <int kN>
__device__ __forceinline__ void write_part(const GradArgs& a, int slot, int col, const float* s) {
  float* p = a.part + (size_t)slot * a.D + col;
#pragma unroll
  for (int e = 0; e < kN; ++e) p[e] = s[e];
}

constexpr int kMaxChunk = 256;

template <typename TG, typename TT, int kN>
__global__ void __launch_bounds__(kThreads, 4) grad_sum_kernel(const GradArgs a) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  __shared__ int s_key[kMaxChunk + 2], s_slot[kMaxChunk];
  const int chunk = blockIdx.x / a.col_tiles, tile = blockIdx.x % a.col_tiles;
  const int p0 = chunk * a.chunk, n = min(a.chunk, a.T - p0);
  for (int i = tid; i < n + 2; i += kThreads) {
    const int p = p0 - 1 + i;
    s_key[i] = p >= 0 && p < a.T ? a.key[p] : -1;
  }
  for (int i = tid; i < n; i += kThreads) s_slot[i] = a.slot[p0 + i];
  __syncthreads();
  const int col = (tile * kThreads + tid) * kN;
  if (col >= a.D) return;
  const TG* g = static_cast<const TG*>(a.grad) + col;
  const int* key = s_key + 1;
  const bool from_before = key[0] == key[-1];        // the first run began in an earlier chunk
  const bool goes_on = key[n - 1] == key[n];         // the last run goes on in the next one
  float acc[kN] = {};
  constexpr int kU = 8;
  bool head = from_before;
  for (int i0 = 0; i0 < n; i0 += kU) {
    Raw<TG, kN> r[kU];
#pragma unroll
    for (int q = 0; q < kU; ++q)
      if (i0 + q < n && key[i0 + q] < a.V)
        r[q] = load_raw<TG, kN>(g + (size_t)s_slot[i0 + q] * a.D);
#pragma unroll
    for (int q = 0; q < kU; ++q) {
      const int i = i0 + q;
      if (i < n && key[i] < a.V) {
        float v[kN];
        expand<TG, kN>(r[q], v);
#pragma unroll
        for (int e = 0; e < kN; ++e) acc[e] += v[e];
        const bool last = i == n - 1;
        if (last || key[i + 1] != key[i]) {
          if (head) write_part<kN>(a, 2 * chunk, col, acc);
          else if (last && goes_on) write_part<kN>(a, 2 * chunk + 1, col, acc);
          else write_row<TT, kN>(a, key[i], col, acc);
          head = false;
#pragma unroll
          for (int e = 0; e < kN; ++e) acc[e] = 0.f;
        }
      }
    }
  }
}

// Joins the partial rows of the runs that cross chunk ends: the run that begins in chunk c and
// goes on behind it is the tail row of c plus the head rows of the chunks behind, in order.
// A CTA takes 32 columns and every gridDim.y-th chunk; its 16 groups of 32 threads take the
// short runs one each, and a long run together, in consecutive shares joined in order.
constexpr int kJoinGroups = 16, kJoinCols = 32, kJoinThreads = kJoinGroups * kJoinCols;
constexpr int kJoinFirst = 2048;
constexpr int kJoinAlone = 16;  // head rows that one group adds by itself

template <typename TT>
__global__ void __launch_bounds__(kJoinThreads) grad_join_kernel(const GradArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int s_chunk[kJoinThreads], s_heads[kJoinThreads], s_count;
  __shared__ int s_first[kJoinFirst];  // the chunks' first tokens
  __shared__ float s[kJoinGroups][kJoinCols];
  const int x = threadIdx.x % kJoinCols, y = threadIdx.x / kJoinCols;
  const int col = blockIdx.x * kJoinCols + x;
  const int step = gridDim.y;
  const bool near = a.chunks <= kJoinFirst;
  if (near)
    for (int c = threadIdx.x; c < a.chunks; c += kJoinThreads) s_first[c] = a.key[c * a.chunk];
  for (int c0 = blockIdx.y; c0 < a.chunks; c0 += step * kJoinThreads) {
    __syncthreads();
    if (threadIdx.x == 0) s_count = 0;
    __syncthreads();
    const int chunk = c0 + (int)threadIdx.x * step;
    const long p0 = (long)chunk * a.chunk, p1 = p0 + a.chunk;
    if (chunk < a.chunks && p1 < a.T) {
      const int v = a.key[p1 - 1];
      if (v < a.V && a.key[p1] == v && (p0 == 0 || a.key[p0 - 1] != v)) {
        int lo = chunk + 1, hi = a.chunks;  // the first chunk that begins behind the run
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if ((near ? s_first[mid] : a.key[(size_t)mid * a.chunk]) <= v) lo = mid + 1;
          else hi = mid;
        }
        const int at = atomicAdd(&s_count, 1);
        s_chunk[at] = chunk;
        s_heads[at] = lo - 1 - chunk;  // chunks behind that begin with the run
      }
    }
    __syncthreads();
    const int count = s_count;
    for (int i = y; i < count; i += kJoinGroups) {
      const int c = s_chunk[i], heads = s_heads[i];
      if (heads > kJoinAlone || col >= a.D) continue;
      float acc = a.part[(size_t)(2 * c + 1) * a.D + col];
      for (int h = 1; h <= heads; ++h) acc += a.part[(size_t)(2 * (c + h)) * a.D + col];
      write_row<TT, 1>(a, a.key[(size_t)(c + 1) * a.chunk], col, &acc);
    }
    for (int i = 0; i < count; ++i) {
      const int c = s_chunk[i], heads = s_heads[i];
      if (heads <= kJoinAlone) continue;
      const int share = (heads + kJoinGroups - 1) / kJoinGroups;
      const int h1 = min(heads, (y + 1) * share);
      float acc = 0.f;
      if (col < a.D) {
        if (y == 0) acc = a.part[(size_t)(2 * c + 1) * a.D + col];
#pragma unroll 8
        for (int h = y * share; h < h1; ++h)
          acc += a.part[(size_t)(2 * (c + 1 + h)) * a.D + col];
      }
      __syncthreads();
      s[y][x] = acc;
      __syncthreads();
      if (y == 0 && col < a.D) {
        for (int k = 1; k < kJoinGroups; ++k) acc += s[k][x];
        write_row<TT, 1>(a, a.key[(size_t)(c + 1) * a.chunk], col, &acc);
      }
    }
  }
}

// Chunk of sorted slots per CTA: about eight CTAs of sums per SM, 16 to 256 slots (a shorter
// chunk writes more partial rows, a longer one leaves SMs idle and is one long chain of loads:
// 32768 slots x 1024 take 73 us in chunks of 16, 92 of 64, 209 of 256; 65536 x 64 take 71, 64
// and 123).
int chunk_len(int T, int D, int sms) {
  const long tiles = (D + 2047) / 2048;
  long c = ((long)T * tiles + 8L * sms - 1) / (8L * sms);
  c = (c + 15) / 16 * 16;
  return (int)(c < 16 ? 16 : c > kMaxChunk ? kMaxChunk : c);
}

}  // namespace

EmbedGradLayout embed_grad_layout(int V, int D, int T, int sms, void* ws) {
  EmbedGradLayout l;
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* p = base ? base + l.bytes : nullptr;
    l.bytes += (bytes + 255) / 256 * 256;
    return p;
  };
  l.chunk = chunk_len(T, D, sms);
  l.chunks = (int)(((long)T + l.chunk - 1) / l.chunk);  // T up to 2^31 - 1
  l.key[0] = reinterpret_cast<int32_t*>(take((size_t)T * 4));
  l.slot[0] = reinterpret_cast<int32_t*>(take((size_t)T * 4));
  if (T > kRankMax) {
    l.tiles = (int)(((long)T + kTile - 1) / kTile);
    l.key[1] = reinterpret_cast<int32_t*>(take((size_t)T * 4));
    l.slot[1] = reinterpret_cast<int32_t*>(take((size_t)T * 4));
    l.hist = reinterpret_cast<uint32_t*>(take((size_t)l.tiles * kDigits * 4));
    for (long v = V; v > 0; v >>= kDigitBits) ++l.passes;  // keys 0 .. V
  }
  l.part = reinterpret_cast<float*>(take((size_t)2 * l.chunks * D * 4));
  return l;
}

int embed_grad_launches(const EmbedGradLayout& l) {
  if (l.chunks == 0) return 1;
  return (l.passes ? 3 * l.passes : 1) + 1 + (l.chunks > 1 ? 1 : 0);
}

cudaError_t launch_embed(const void* table, int dtype, int V, int D, const int32_t* ids, int T,
                         float scale, void* out, int sms, unsigned* status, cudaStream_t stream) {
  const size_t elem = dtype == DFLASH_DTYPE_BF16 ? 2 : 4;
  const bool vec = (size_t)D * elem % 16 == 0;
  const int nvec = vec ? (int)((size_t)D * elem / 16) : D;
  int tx = 1;
  while (tx < kThreads && tx * kHold < nvec) tx *= 2;
  const int cols = (nvec + kHold * tx - 1) / (kHold * tx);
  // 16 slots per row of threads, fewer while that leaves SMs without a CTA or two
  const int ny = kThreads / tx;
  int rows = 16 * ny;
  auto ctas = [&]() { return ((long)T + rows - 1) / rows; };
  while (rows > 1 && ctas() * cols < 2L * sms) rows /= 2;
  if (rows > kMaxRows) rows = kMaxRows;
  const dim3 grid((unsigned)ctas(), (unsigned)cols);
  auto go = [&](auto kernel, auto* t) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(t)>>;
    return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, t, V, D, ids, T, scale,
                      static_cast<E*>(out), tx, rows, status);
  };
  if (dtype == DFLASH_DTYPE_BF16) {
    const auto* t = static_cast<const __nv_bfloat16*>(table);
    return vec ? go(embed_kernel<__nv_bfloat16, 8>, t) : go(embed_kernel<__nv_bfloat16, 1>, t);
  }
  const auto* t = static_cast<const float*>(table);
  return vec ? go(embed_kernel<float, 4>, t) : go(embed_kernel<float, 1>, t);
}

namespace {

template <typename TG, typename TT, int kN>
cudaError_t launch_sums(GradArgs a, cudaStream_t stream) {
  a.col_tiles = (a.D + kThreads * kN - 1) / (kThreads * kN);
  cudaError_t e = launch_pdl(grad_sum_kernel<TG, TT, kN>,
                             dim3((unsigned)(a.chunks * a.col_tiles)), dim3(kThreads), 0, stream,
                             a);
  if (e != cudaSuccess || a.chunks < 2) return e;
  return launch_pdl(grad_join_kernel<TT>,
                    dim3((unsigned)((a.D + kJoinCols - 1) / kJoinCols),
                         (unsigned)(a.chunks < 8 ? a.chunks : 8)),
                    dim3(kJoinThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_embed_grad(const void* grad, int grad_dtype, const int32_t* ids, int T, int V,
                              int D, float scale, bool accumulate, void* table, int table_dtype,
                              const EmbedGradLayout& l, int sms, unsigned* status,
                              cudaStream_t stream) {
  cudaError_t e;
  int cur = 0;
  Fill fill = {table, 0};
  if (!accumulate) fill.bytes = (size_t)V * D * (table_dtype == DFLASH_DTYPE_BF16 ? 2 : 4);
  // CTAs for the zeros: 64 KB each at least, at most 8 per SM
  long fills = (long)((fill.bytes + 65535) / 65536);
  if (fills > 8L * sms) fills = 8L * sms;
  if (T == 0 || l.passes == 0) {
    const unsigned ctas = (unsigned)((T + 63) / 64);
    e = launch_pdl(rank_kernel, dim3(ctas + (unsigned)fills), dim3(512), 0, stream, ids, T, V,
                   l.key[0], l.slot[0], ctas, fill, status);
    if (e != cudaSuccess || T == 0) return e;
  } else {
    const int32_t *key = nullptr, *slot = nullptr;
    for (int p = 0; p < l.passes; ++p) {
      const int shift = p * kDigitBits;
      cur = p & 1;
      e = launch_pdl(radix_count_kernel, dim3((unsigned)(l.tiles + (p ? 0 : fills))),
                     dim3(kThreads), 0, stream, key, ids, T, V, shift, l.tiles, l.hist, fill,
                     status);
      if (e != cudaSuccess) return e;
      e = launch_pdl(radix_scan_kernel, dim3(1), dim3(1024), 0, stream, l.hist,
                     l.tiles * kDigits);
      if (e != cudaSuccess) return e;
      e = launch_pdl(radix_scatter_kernel, dim3((unsigned)l.tiles), dim3(kThreads), 0, stream,
                     key, slot, ids, T, V, shift, l.tiles, l.hist, l.key[cur], l.slot[cur],
                     status);
      if (e != cudaSuccess) return e;
      key = l.key[cur];
      slot = l.slot[cur];
    }
  }
  GradArgs a = {};
  a.grad = grad;
  a.key = l.key[cur];
  a.slot = l.slot[cur];
  a.T = T;
  a.V = V;
  a.D = D;
  a.scale = scale;
  a.accumulate = accumulate ? 1 : 0;
  a.table = table;
  a.part = l.part;
  a.chunk = l.chunk;
  a.chunks = l.chunks;
  const bool gb = grad_dtype == DFLASH_DTYPE_BF16, tb = table_dtype == DFLASH_DTYPE_BF16;
  const bool vec = D % (gb ? 8 : 4) == 0;  // 16-byte rows of grad, rows of table aligned to a pack
  if (gb) {
    if (tb)
      return vec ? launch_sums<__nv_bfloat16, __nv_bfloat16, 8>(a, stream)
                 : launch_sums<__nv_bfloat16, __nv_bfloat16, 1>(a, stream);
    return vec ? launch_sums<__nv_bfloat16, float, 8>(a, stream)
               : launch_sums<__nv_bfloat16, float, 1>(a, stream);
  }
  if (tb)
    return vec ? launch_sums<float, __nv_bfloat16, 4>(a, stream)
               : launch_sums<float, __nv_bfloat16, 1>(a, stream);
  return vec ? launch_sums<float, float, 4>(a, stream) : launch_sums<float, float, 1>(a, stream);
}

}  // namespace dflash
