// The kernel of a filtered row (sample.cuh describes it), for the files that compile it.
#pragma once

#include "sample.cuh"

namespace dflash {

namespace {

// kVerify: writes the row's statistics and its proposal's acceptance; else samples it.
template <typename T, bool kVerify, int kNT>
__global__ void __launch_bounds__(kNT, 1024 / kNT) filter_kernel(const FilterArgs a) {
  __shared__ Shared sh;
  constexpr int kN = Slice<T, kNT>::kN, kWarps = kNT / 32, kKeys = kList / kNT;
  constexpr float kLowest = -3.402823466e38f;
  pdl_wait();
  pdl_trigger();
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.C;
  const int rank = (int)(blockIdx.x % (unsigned)C);
  const int row = (int)(blockIdx.x / (unsigned)C);
  const int V = a.V;
  const int req = row / a.per;
  const T* lrow = static_cast<const T*>(a.logits) + (size_t)row * a.ld;

  const int len = ((V + C - 1) / C + 7) / 8 * 8;
  Slice<T, kNT> sl;
  sl.init(lrow, min(V, rank * len), min(V, (rank + 1) * len));

  auto fill_zero = [&]() {
    float* out = a.probs + (size_t)row * V;
    const int i = sl.c0;
    const int mis = (int)(((uintptr_t)(out + i) & 15) / 4);
    const int head = min(sl.c1, i + (mis ? 4 - mis : 0));
    for (int x = i + tid; x < head; x += kNT) out[x] = 0.f;
    const int n4 = (sl.c1 - head) / 4;
    float4* o4 = reinterpret_cast<float4*>(out + head);
    for (int x = tid; x < n4; x += kNT) o4[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = head + 4 * n4 + tid; x < sl.c1; x += kNT) out[x] = 0.f;
  };
  // a row that keeps nothing
  auto finish_empty = [&]() {
    if constexpr (kVerify) {
      if (rank == 0 && tid == 0) {
        RowStats st = {};
        st.mx = -INFINITY;
        a.stats[row] = st;
        a.accept[row] = 0;
      }
    } else {
      if (a.probs) fill_zero();
      if (rank == 0 && tid == 0) a.tokens[row] = -1;
    }
  };
  // ---- this row's settings, and the slice's largest logits ----
  const float temp = a.temperature ? a.temperature[req] : 1.f;
  const int top_k = a.top_k ? a.top_k[req] : 0;
  const float top_p = a.top_p ? a.top_p[req] : 1.f;
  const float min_p = a.min_p ? a.min_p[req] : 0.f;
  const float u = kVerify ? (row % a.per < a.gamma ? a.uniforms[row] : 0.f) : a.uniforms[row];
  if (tid < 32) {
    sh.tab.fix[tid] = kExp2Table[tid];
    sh.tab.flt[tid] = (float)kExp2Table[tid];
  }
  if (tid == 0) sh.list_n = 0;
  float tmax = -INFINITY;  // a NaN is dropped
  int jmax = 0;            // greedy: the first vector that holds tmax
  if (temp == 0.f) {
    sl.template each<8>([&](int j, const uint4& r) {
      const float m = Vec<T>::largest(r);
      if (m > tmax) {
        tmax = m;
        jmax = j;
      }
    });
  } else {
    typename Vec<T>::Max running;
    sl.template each<8>([&](int, const uint4& x) { running.push(x); });
    tmax = running.value();
  }
  const bool ok = (temp == 0.f || (temp >= kMinTemp && temp <= kMaxTemp)) && top_k >= 0 &&
                  top_p > 0.f && top_p <= 1.f && min_p >= 0.f && min_p <= 1.f && u >= 0.f &&
                  u < 1.f;
  if (!ok) {  // the same in every CTA of the cluster, before any of them waits
    if (tid == 0 && rank == 0) report(a.status, kStatusCheck, kKernSample);
    finish_empty();
    return;
  }
  cl.barrier_arrive();  // waited for below: no CTA writes into one that has not started

  const bool use_k = top_k > 0 && top_k < V && temp > 0.f;
  const bool use_m = min_p > 0.f && temp > 0.f;
  const bool use_p = top_p < 1.f && temp > 0.f;
  // A value that at least `tokens` tokens of the row reach: the m-th largest of the maxima of
  // groups of this CTA's threads, m = tokens / C rounded up -- the smallest of the CTAs'
  // values.  The more of the groups it takes, the more tokens reach it beyond those: at
  // three quarters of them about 1.85 times as many.
  const int tokens = use_k ? top_k : use_p && !use_m ? min(kGuess, V) : 0;
  const int m = (tokens + C - 1) / C;
  // 2^glog threads per group
  const int glog = m <= 48 ? (kNT == 512 ? 3 : 2) : m <= 96 && kNT == 512 ? 2 : 0;
  const int groups = kNT >> glog;
  const bool by_maxima = tokens > 0 && m <= kNT / 8 * 7 && tokens <= kList / 2;
  float gm = tmax;
  for (int o = 1; o < 1 << glog; o <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  if ((lane & ((1 << glog) - 1)) == 0) sh.gmax[tid >> glog] = gm;
  if (tid == 0) sh.cthr[rank] = kLowest;
  __syncthreads();
  float mx = -INFINITY;
  const float4* g4 = reinterpret_cast<const float4*>(sh.gmax);
  for (int i = lane; i < groups / 4; i += 32) {
    const float4 g = g4[i];
    mx = fmaxf(fmaxf(mx, fmaxf(g.x, g.y)), fmaxf(g.z, g.w));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (by_maxima) {
    const int per = 1 << glog, mine = tid >> glog;  // per threads count for a group
    const float v = sh.gmax[mine];
    int n = 0;
    for (int i = tid & (per - 1); i < groups / 4; i += per) {
      const float4 g = g4[i];
      n += (g.x > v || (g.x == v && 4 * i < mine)) + (g.y > v || (g.y == v && 4 * i + 1 < mine)) +
           (g.z > v || (g.z == v && 4 * i + 2 < mine)) +
           (g.w > v || (g.w == v && 4 * i + 3 < mine));
    }
    for (int o = 1; o < per; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (n == m - 1) sh.cthr[rank] = fmaxf(v, kLowest);
    __syncthreads();
  }
  // chi + clo = log2(e) / T to about 2^-46
  float chi = 0.f, clo = 0.f;
  if (temp > 0.f) {
    chi = __fdiv_rn(1.44269502f, temp);
    clo = __fdiv_rn(fmaf(-chi, temp, 1.44269502f) + 1.92596299e-8f, temp);
  }
  cl.barrier_wait();
  publish(cl, sh.cmax, rank, C, mx);
  if (by_maxima && tid < C && tid != rank) cl.map_shared_rank(sh.cthr, tid)[rank] = sh.cthr[rank];
  cl.sync();
  float guess = by_maxima ? INFINITY : kLowest;
#pragma unroll
  for (int r = 0; r < kMaxC; ++r) {
    if (r < C) {
      mx = fmaxf(mx, sh.cmax[r]);
      if (by_maxima) guess = fminf(guess, sh.cthr[r]);
    }
  }
  if (mx == -INFINITY) {
    finish_empty();
    return;  // no CTA touches another's shared memory after the barrier above
  }
  // without min_p every finite logit passes
  const float thr = use_m ? min_p_threshold(mx, temp, min_p, sh.tab) : kLowest;
  const bool fast_ok = fabsf(mx) < kFastLogit;
  float pivot = mx == INFINITY ? mx : thr;  // +inf entries share everything
  int cut = 0x7fffffff;
  float above_pivot = INFINITY;  // the next float up, once there is a cut
  auto kept = [&](float l, int i) { return l > pivot || (l == pivot && i <= cut); };
  // The least value that a kept token among the indices i0 .. i0 + kN - 1 has: all of them lie
  // on one side of `cut`, or (NaN) they have to be looked at one by one.
  auto least_kept = [&](int i0) -> float {
    if (i0 + kN - 1 <= cut) return pivot;
    return i0 > cut ? above_pivot : NAN;
  };
  const float sb = 32.f * chi;
  auto bucket = [&](float l) {
    const float d = l == mx ? 0.f : mx - l;
    return __float2int_rz(fminf(d * sb, (float)(kBuckets - 1)));
  };
  auto units = [&](float l) { return weight_units(l, mx, chi, clo, sh.tab); };

  u64 z = 0;        // kept mass
  int token = -2;
  bool listed = false;
  int list_n = 0;       // CTA 0: tokens in list.key, and the last kept one in their order
  u64 list_last = 0;
  const int kPlaces = min(kList, kSlots / C);

  // Gathers the tokens >= lo for which pred holds in CTA 0; their number in the row, more than
  // kList if they do not all have a place (`places` for each CTA).  also(vector) is added up
  // over the row into *sum.
  auto gather = [&](float lo, int places, auto pred, auto also, u64* sum) -> int {
    u64* slot = cl.map_shared_rank(sh.list.slot, 0) + rank * (kSlots / C);
    u64 mine = 0;
    const typename Vec<T>::AtLeast test(lo);
    sl.template each<4>([&](int j, const uint4& r) {
      mine += also(r);
      if (!test.any(r)) return;
      float v[kN];
      Vec<T>::unpack(r, v);
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const int i = sl.first + j * kN + e;
        if (v[e] >= lo && pred(v[e], i)) {
          const uint32_t at = atomicAdd(&sh.list_n, 1u);
          if (at < (uint32_t)places) slot[at] = (u64)desc_key(v[e]) << 32 | (uint32_t)i;
        }
      }
    });
    mine = warp_sum64(mine);
    if (lane == 0) sh.warp64[warp] = mine;
    __syncthreads();
    if (tid < C) {
      u64 t = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += sh.warp64[w];
      cl.map_shared_rank(sh.clist, tid)[rank] = sh.list_n;
      cl.map_shared_rank(sh.cmass, tid)[rank] = t;
    }
    cl.sync();
    if (tid == 0) sh.list_n = 0;
    int n = 0;
    u64 t = 0;
#pragma unroll
    for (int r = 0; r < kMaxC; ++r) {
      if (r < C) {
        const int c = (int)min(sh.clist[r], 1u << 20);
        n += c <= places ? c : kList + 1;
        t += sh.cmass[r];
      }
    }
    *sum = t;
    return n;
  };
  auto all = [](float, int) { return true; };
  auto nothing = [](const uint4&) { return 0ull; };
  // CTA 0: gathered token i (~0 behind the last)
  auto gathered = [&](uint32_t i) -> u64 {
#pragma unroll
    for (int r = 0; r < kMaxC; ++r) {
      if (r < C) {
        const uint32_t n = sh.clist[r];
        if (i < n) return sh.list.slot[r * (kSlots / C) + i];
        i -= n;
      }
    }
    return ~0ull;
  };
  // ... kKeys per thread
  auto pull = [&](u64 (&k)[kKeys]) {
#pragma unroll
    for (int q = 0; q < kKeys; ++q) k[q] = gathered(tid + q * kNT);
  };
  // inclusive masses of the first n sorted tokens into list.mass; the weights in w
  auto list_masses = [&](const u64 (&k)[kKeys], int n, u64 (&w)[kKeys], bool by_index) {
    u64 base = 0;
#pragma unroll
    for (int q = 0; q < kKeys; ++q) {
      if (q * kNT >= n) break;
      const int i = tid + q * kNT;
      w[q] = i < n ? units(key_value((uint32_t)(by_index ? k[q] : k[q] >> 32))) : 0;
      u64 m = w[q], mt;
      uint32_t c = 0, ct;
      block_scan<kNT>(c, m, ct, mt, sh);
      if (i < n) sh.list.mass[i] = base + m;
      base += mt;
    }
    __syncthreads();
  };

  // CTA 0 finishes the row from its n gathered tokens, a superset of the kept ones.  z_all: the
  // mass that top_p refers to, with the relative error of fast sums (fast); else top_p refers
  // to the list's mass after top_k.  False: a border of top_p lies within that error, or
  // behind the list.
  //
  // Few tokens: kNT / 2^ceil(log2 n) threads per token count the tokens before it in the
  // sorted order, which gives its place; then, among the kept, add the mass before it in
  // index order.
  auto count_list = [&](int n, u64 z_all, bool fast) -> bool {
    int lg = 4;
    while (1 << lg < n) ++lg;
    const int per_lg = (kNT == 512 ? 9 : 8) - lg, per = 1 << per_lg;
    const int i = tid >> per_lg, part = tid & (per - 1);
    if (tid < n) {
      const u64 k = gathered(tid);
      sh.list.key[tid] = k;
      sh.list.mass[tid] = units(key_value((uint32_t)(k >> 32)));
    }
    if (tid == 0) sh.verdict = 0;
    __syncthreads();
    const bool in = i < n;
    const u64 key = in ? sh.list.key[i] : ~0ull, w = in ? sh.list.mass[i] : 0;
    int at = 0;
#pragma unroll 4
    for (int j = part; j < n; j += per) at += sh.list.key[j] < key ? 1 : 0;
    for (int o = 1; o < per; o <<= 1) at += __shfl_xor_sync(0xffffffffu, at, o);
    __syncthreads();
    if (in && part == 0) {
      sh.list.key[at] = key;
      sh.list.mass[at] = w;
    }
    __syncthreads();
    int keep = use_k && top_k < n ? top_k : n;
    if (warp == 0) {
      // the mass up to each token; the last that top_p keeps: without it the mass is short
      constexpr int kPer = kCountList / 32;
      u64 m[kPer], sum = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int j = lane * kPer + e;
        m[e] = sum += j < keep ? sh.list.mass[j] : 0;
      }
      u64 incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const u64 total = __shfl_sync(0xffffffffu, incl, 31);
      u64 need = total, err = 0;
      if (use_p) {
        need = share_of(top_p, fast ? z_all : total);
        if (fast) err = (need >> kRoughBits) + 1;
      }
      u64 before = incl - sum;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int j = lane * kPer + e;
        const u64 upto = incl - sum + m[e];
        if (j < keep && (use_p ? before < need && upto >= need : j == keep - 1)) {
          sh.last_key = sh.list.key[j];
          sh.last_z = upto;
          sh.index = j + 1;
          sh.verdict = !use_p || ((before + err < need || j == 0) && upto >= need + err);
        }
        before = upto;
      }
    }
    __syncthreads();
    if (!sh.verdict) return false;
    keep = sh.index;
    list_n = keep;
    list_last = sh.last_key;
    z = sh.last_z;
    if constexpr (!kVerify) {
      const u64 t = mul_fraction(u, z, false);
      for (int i0 = 0; i0 < keep; i0 += kNT >> per_lg) {
        const int x = i0 + i;
        const bool is = x < keep;
        const u64 key2 = is ? sh.list.key[x] : 0, w2 = is ? sh.list.mass[x] : 0;
        u64 c = 0;
#pragma unroll 4
        for (int j = part; j < keep; j += per) {
          const u64 m = sh.list.mass[j];
          c += (uint32_t)sh.list.key[j] < (uint32_t)key2 ? m : 0;
        }
        for (int o = 1; o < per; o <<= 1) c += shfl_xor64(c, o);
        if (is && part == 0 && c <= t && t - c < w2) sh.warpi[0] = (int)(uint32_t)key2;
      }
      __syncthreads();
      token = sh.warpi[0];
    }
    return true;
  };
  auto sort_list = [&](int n, u64 z_all, bool fast) -> bool {
    u64 k[kKeys], w[kKeys];
    pull(k);
    sort_keys<kNT>(sh, k, n);
    int keep = use_k && top_k < n ? top_k : n;
    list_masses(k, keep, w, false);
    if (use_p) {
      const u64 need = share_of(top_p, fast ? z_all : sh.list.mass[keep - 1]);
      const u64 err = fast ? (need >> kRoughBits) + 1 : 0;
      if (tid == 0) {
        sh.index = keep;
        sh.verdict = fast ? 0 : 1;
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kKeys; ++q) {
        const int i = tid + q * kNT;
        if (i < keep) {
          const u64 incl = sh.list.mass[i], before = incl - w[q];
          if (before < need && incl >= need) {
            sh.index = i + 1;
            if (fast && (before + err < need || i == 0) && incl >= need + err) sh.verdict = 1;
          }
        }
      }
      __syncthreads();
      keep = sh.index;
      if (!sh.verdict) return false;
    }
    z = sh.list.mass[keep - 1];
    list_n = keep;
    list_last = sh.list.key[keep - 1];
    if constexpr (!kVerify) {
      // the kept tokens by index
      u64 by[kKeys];
#pragma unroll
      for (int q = 0; q < kKeys; ++q)
        by[q] = tid + q * kNT < keep ? k[q] << 32 | k[q] >> 32 : ~0ull;
      sort_keys<kNT>(sh, by, keep);
      list_masses(by, keep, w, true);
      const u64 t = mul_fraction(u, z, false);
#pragma unroll
      for (int q = 0; q < kKeys; ++q) {
        const int i = tid + q * kNT;
        if (i < keep) {
          const u64 incl = sh.list.mass[i];
          if (incl > t && incl - w[q] <= t && w[q]) sh.index = (int)(by[q] >> 32);
          sh.list.key[i] = k[q];
        }
      }
      __syncthreads();
      token = sh.index;
    }
    return true;
  };
  // The row from its n gathered tokens; false: undecided within the error of fast sums.  Ends
  // with the row's zeros written before CTA 0 goes on.
  auto from_list = [&](int n, u64 z_all, bool fast) -> bool {
    const bool zeros = !kVerify && a.probs;
    bool good = true;
    if (rank == 0) {
      if (fast && n > kCountList) {  // most rows that keep more tokens show it by the list's mass
        u64 k[kKeys], m = 0, mt;
        uint32_t c = 0, ct;
        pull(k);
#pragma unroll
        for (int q = 0; q < kKeys; ++q)
          if (tid + q * kNT < n) m += units(key_value((uint32_t)(k[q] >> 32)));
        block_scan<kNT>(c, m, ct, mt, sh);
        good = mt >= share_of(top_p, z_all);
      }
      if (zeros) fill_zero();
      if (good) good = n <= kCountList ? count_list(n, z_all, fast) : sort_list(n, z_all, fast);
      if (good) {
        pivot = key_value((uint32_t)(list_last >> 32));
        cut = (int)(uint32_t)list_last;
      }
      if (fast && tid < C) *cl.map_shared_rank(&sh.verdict, tid) = good ? 1 : 0;
    } else if (zeros) {
      fill_zero();
    }
    if (fast || zeros) cl.sync();
    if (fast) good = sh.verdict != 0;
    return good;
  };

  // joins a value of each CTA: their sum
  auto cluster_sum = [&](u64 v) -> u64 {
    u64 m = v, mt, total = 0;
    uint32_t c = 0, ct;
    block_scan<kNT>(c, m, ct, mt, sh);
    publish(cl, sh.cmass, rank, C, mt);
    cl.sync();
    for (int r = 0; r < C; ++r) total += sh.cmass[r];
    return total;
  };

  // Joins the CTAs' histograms -- counts, and masses (by_mass: the pieces; else low(bucket)
  // per token) -- and finds the bucket in which the count reaches k, or the mass reaches
  // need(total mass).  bucket = kBuckets: neither is reached.
  auto join = [&](bool by_mass, auto low, uint32_t k, auto need_of) {
    cl.sync();
    const int seg = kBuckets / C;            // CTA `rank` joins buckets [rank * seg, ...)
    const int bpt = (seg + kNT - 1) / kNT;   // buckets per thread, consecutive
    constexpr int kMost = kBuckets / kNT;    // of them
    uint32_t bc[kMost] = {};
    u64 bm[kMost] = {};
    uint32_t tc = 0;
    u64 tm = 0;
    for (int i = 0; i < bpt; ++i) {
      const int b = tid * bpt + i;
      if (b < seg) {
        for (int r = 0; r < C; ++r) {
          const uint32_t* h = cl.map_shared_rank(&sh.hist[0][0], r) + rank * seg + b;
          bc[i] += h[0];
          if (by_mass)
            bm[i] += (u64)h[kBuckets] + ((u64)h[2 * kBuckets] << 15) + ((u64)h[3 * kBuckets] << 30);
        }
        if (!by_mass) bm[i] = bc[i] * low(rank * seg + b);
      }
      tc += bc[i];
      tm += bm[i];
    }
    uint32_t ic = tc, ctot;
    u64 im = tm, mtot;
    block_scan<kNT>(ic, im, ctot, mtot, sh);
    publish(cl, sh.ccnt, rank, C, ctot);
    publish(cl, sh.cmass, rank, C, mtot);
    if (tid == 0) sh.found.bucket = kBuckets;
    cl.sync();
    uint32_t call = 0, cbefore = 0;
    u64 mall = 0, mbefore = 0;
    for (int r = 0; r < C; ++r) {
      if (r == rank) {
        cbefore = call;
        mbefore = mall;
      }
      call += sh.ccnt[r];
      mall += sh.cmass[r];
    }
    const u64 need = need_of(mall);
    uint32_t c0 = cbefore + ic - tc;
    u64 m0 = mbefore + im - tm;
    for (int i = 0; i < bpt; ++i) {
      const bool cross = k ? (c0 < k && c0 + bc[i] >= k) : (m0 < need && m0 + bm[i] >= need);
      if (cross) {  // the thread in whose buckets the crossing lies tells every CTA
        Shared::Found f;
        f.bucket = rank * seg + tid * bpt + i;
        f.cnt_before = c0;
        f.cnt_in = bc[i];
        f.mass_before = m0;
        f.total = mall;
        for (int r = 0; r < C; ++r) *cl.map_shared_rank(&sh.found, r) = f;
      }
      c0 += bc[i];
      m0 += bm[i];
    }
    cl.sync();
    Shared::Found f = sh.found;
    if (f.bucket == kBuckets) {
      f.cnt_before = call;
      f.cnt_in = 0;
      f.mass_before = f.total = mall;
    }
    return f;
  };
  auto no_low = [](int) { return 0ull; };
  auto no_need = [](u64) { return 0ull; };

  // Histogram of the kept tokens by count, or by mass.
  auto histogram = [&](bool by_mass) {
    for (int i = tid; i < (by_mass ? 4 : 1) * kBuckets; i += kNT) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    sl.template each<2>([&](int j, const uint4& r) {
      float v[kN];
      Vec<T>::unpack(r, v);
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        if (!kept(v[e], sl.first + j * kN + e)) continue;
        const int b = bucket(v[e]);
        atomicAdd(&sh.hist[0][b], 1u);
        if (by_mass) {
          const u64 w = units(v[e]);
          const uint32_t p0 = (uint32_t)w & 0x7fffu, p1 = (uint32_t)(w >> 15) & 0x7fffu,
                         p2 = (uint32_t)(w >> 30);
          if (p0) atomicAdd(&sh.hist[1][b], p0);
          if (p1) atomicAdd(&sh.hist[2][b], p1);
          if (p2) atomicAdd(&sh.hist[3][b], p2);
        }
      }
    });
  };

  // The pivot inside the bucket f.bucket: the token at which the count reaches want, or the
  // mass reaches need, counted from the bucket's start.
  auto cut_bucket = [&](const Shared::Found& f, bool by_mass, uint32_t want, u64 need) {
    const int jb = f.bucket;
    if (f.cnt_in <= (uint32_t)kPlaces) {
      u64 none;
      gather(kLowest, kPlaces, [&](float l, int i) { return kept(l, i) && bucket(l) == jb; },
             nothing, &none);
      if (rank == 0) {
        const int n = (int)f.cnt_in;
        u64 k[kKeys], w[kKeys];
        pull(k);
        sort_keys<kNT>(sh, k, n);
        if (by_mass) list_masses(k, n, w, false);
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
          const int i = tid + q * kNT;
          if (i < n) {
            bool here = (uint32_t)i == want - 1;
            if (by_mass) {
              const u64 incl = sh.list.mass[i];
              here = incl >= need && incl - w[q] < need;
            }
            if (here) {
              Shared::Pivot p;
              p.value = key_value((uint32_t)(k[q] >> 32));
              p.cut = (int)(uint32_t)k[q];
              for (int r = 0; r < C; ++r) *cl.map_shared_rank(&sh.pivot, r) = p;
            }
          }
        }
      }
      cl.sync();
      pivot = sh.pivot.value;
      cut = sh.pivot.cut;
      return;
    }
    // radix selection on the logit's bits, 8 at a time, then the index among equal logits
    uint32_t prefix = 0, mask = 0;
    uint32_t c_left = want;
    u64 m_left = need;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 4 * 256; i += kNT) (&sh.hist[0][0])[i] = 0;
      __syncthreads();
      uint32_t* h = &sh.hist[0][0];
      for (int j = tid; j < sl.nv; j += kNT) {
        float v[kN];
        sl.values(j, v);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          if (!kept(v[e], sl.first + j * kN + e) || bucket(v[e]) != jb) continue;
          const uint32_t key = desc_key(v[e]);
          if ((key & mask) != prefix) continue;
          const int b = key >> shift & 255;
          atomicAdd(&h[b], 1u);
          if (by_mass) {
            const u64 w = units(v[e]);
            const uint32_t p0 = (uint32_t)w & 0x7fffu, p1 = (uint32_t)(w >> 15) & 0x7fffu,
                           p2 = (uint32_t)(w >> 30);
            if (p0) atomicAdd(&h[256 + b], p0);
            if (p1) atomicAdd(&h[512 + b], p1);
            if (p2) atomicAdd(&h[768 + b], p2);
          }
        }
      }
      cl.sync();
      uint32_t bc = 0;
      u64 bm = 0;
      if (tid < 256) {
        for (int r = 0; r < C; ++r) {
          const uint32_t* hr = cl.map_shared_rank(&sh.hist[0][0], r) + tid;
          bc += hr[0];
          bm += (u64)hr[256] + ((u64)hr[512] << 15) + ((u64)hr[768] << 30);
        }
      }
      uint32_t ic = bc, ctot;
      u64 im = bm, mtot;
      block_scan<kNT>(ic, im, ctot, mtot, sh);
      const bool cross = by_mass ? (im - bm < m_left && im >= m_left)
                                 : (ic - bc < c_left && ic >= c_left);
      if (cross) {   // every CTA finds the same digit for itself
        sh.found.bucket = tid;
        sh.found.cnt_before = ic - bc;
        sh.found.mass_before = im - bm;
      }
      cl.sync();     // also: no CTA clears its histogram while another still reads it
      prefix |= (uint32_t)sh.found.bucket << shift;
      mask |= 255u << shift;
      c_left -= sh.found.cnt_before;
      m_left -= sh.found.mass_before;
      __syncthreads();
    }
    const float pv = key_value(prefix);
    // of the tokens equal to pv, the lowest-index m are kept
    u64 m = c_left;
    if (by_mass) {
      const u64 w = units(pv);
      m = w ? (m_left + w - 1) / w : 1;
    }
    u64 tot;
    const int idx = search<T, kNT>(
        cl, sh, sl, rank, C,
        [&](float l, int i) { return (u64)(l == pv && kept(l, i) ? 1 : 0); },
        [&](u64 t) { return m - 1 < t ? m - 1 : t - 1; }, &tot);
    pivot = pv;
    cut = idx;
  };

  // The cut of bf16 logits by count (k) or by mass (top_p): they take few values, so the tokens
  // are counted per value and a weight is found once per value.  False: the cut lies in a bin
  // of several values.
  // The kept mass comes with it (z).
  // 2 * (magnitude - 2^-9 in bf16 steps) + sign, from a bf16's bits rotated by one; beyond
  // 2 * kValueOctaves for the magnitudes that share a bin
  auto value_index = [](uint32_t word, int half) -> uint32_t {
    const uint32_t r = half ? ((word >> 15) & 0xfffeu) + (word >> 31)
                            : ((word << 1) & 0xfffeu) + ((word >> 15) & 1u);
    return r - 2 * kValueLowest;
  };
  auto bin_index = [](int b) {  // of the bins in order, largest first
    return b <= kValueOctaves ? 2 * (kValueOctaves - b) : 2 * (b - kValueSmall - 1) + 1;
  };
  auto bin_value = [&](int b) {
    const uint32_t m = b <= kValueOctaves ? kValueLowest + kValueOctaves - b
                                          : 0x8000u + kValueLowest + b - kValueSmall - 1;
    return __uint_as_float(m << 16);
  };
  auto value_cut = [&](bool by_mass, uint32_t k) -> bool {
    if constexpr (sizeof(T) != 2) return false;
    const bool some = pivot > kLowest;
    auto& val = sh.val;
    for (int i = tid; i < 2 * kValueOctaves; i += kNT) val.count[i] = 0;
    if (tid < 3) val.mass[tid] = val.zone_count[tid] = 0;
    __syncthreads();
    uint32_t zone_count[3] = {0, 0, 0};
    u64 zone_mass[3] = {0, 0, 0};
    auto several = [&](float l) {  // rare
      const int zone = fabsf(l) < 1.f ? 1 : l < 0.f ? 2 : 0;
      ++zone_count[zone];
      zone_mass[zone] += units(l);
    };
    sl.template each<2>([&](int j, const uint4& r) {
      const uint32_t word[4] = {r.x, r.y, r.z, r.w};
      uint32_t odd = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t c = value_index(word[e >> 1], e & 1);
        const float l = __uint_as_float(e & 1 ? word[e >> 1] & 0xffff0000u : word[e >> 1] << 16);
        const bool in = c < 2 * kValueOctaves;
        odd |= in || !(l >= kLowest) ? 0u : 1u << e;  // -inf and NaN are not kept
        if (in && (!some || kept(l, sl.first + j * 8 + e))) atomicAdd(&val.count[c], 1u);
      }
      // a loop of its own: the weights' code must not run predicated for every token
#pragma unroll 1
      for (; odd; odd &= odd - 1) {
        const int i = sl.first + j * 8 + __ffs(odd) - 1;
        const float l = sl.at(i);
        if (kept(l, i)) several(l);
      }
    });
    for (int i = 0; i < 3; ++i) {
      if (!__any_sync(0xffffffffu, zone_count[i] != 0)) continue;
      const uint32_t c = __reduce_add_sync(0xffffffffu, zone_count[i]);
      const u64 m = warp_sum64(zone_mass[i]);
      if (lane == 0) {
        atomicAdd(&val.zone_count[i], c);
        atomicAdd(&val.mass[i], m);
      }
    }
    cl.sync();
    const int seg = (kValueBins + C - 1) / C;  // CTA `rank` joins bins [rank * seg, ...)
    const int bpt = (seg + kNT - 1) / kNT;
    const int b0 = rank * seg + tid * bpt;
    const int b1 = min(min(b0 + bpt, (rank + 1) * seg), kValueBins);
    auto of_bin = [&](int b, uint32_t& c, u64& m) {
      c = 0;
      m = 0;
      const int s = b == 0 ? 0 : b == kValueSmall ? 1 : b == kValueBins - 1 ? 2 : -1;
      for (int r = 0; r < C; ++r) {
        const auto* o = cl.map_shared_rank(&val, r);
        if (s >= 0) {
          c += o->zone_count[s];
          m += o->mass[s];
        } else {
          c += o->count[bin_index(b)];
        }
      }
      if (s < 0 && c) m = c * units(bin_value(b));
    };
    uint32_t tc = 0, ctot;
    u64 tm = 0, mtot;
    for (int b = b0; b < b1; ++b) {
      uint32_t c;
      u64 m;
      of_bin(b, c, m);
      tc += c;
      tm += m;
    }
    uint32_t ic = tc;
    u64 im = tm;
    block_scan<kNT>(ic, im, ctot, mtot, sh);
    publish(cl, sh.ccnt, rank, C, ctot);
    publish(cl, sh.cmass, rank, C, mtot);
    if (tid == 0) sh.found.bucket = kValueBins;
    cl.sync();
    uint32_t c0 = ic - tc;
    u64 m0 = im - tm, mall = 0;
    for (int r = 0; r < C; ++r) {
      if (r < rank) {
        c0 += sh.ccnt[r];
        m0 += sh.cmass[r];
      }
      mall += sh.cmass[r];
    }
    const u64 need = by_mass ? share_of(top_p, mall) : 0;
    if (by_mass ? m0 < need && m0 + tm >= need : c0 < k && c0 + tc >= k) {
      for (int b = b0; b < b1; ++b) {
        uint32_t c;
        u64 m;
        of_bin(b, c, m);
        if (by_mass ? m0 < need && m0 + m >= need : c0 < k && c0 + c >= k) {
          Shared::Found f;
          f.bucket = b;
          f.cnt_before = c0;
          f.cnt_in = c;
          f.mass_before = m0;
          f.total = mall;
          for (int r = 0; r < C; ++r) *cl.map_shared_rank(&sh.found, r) = f;
        }
        c0 += c;
        m0 += m;
      }
    }
    cl.sync();
    const Shared::Found f = sh.found;
    if (f.bucket == kValueBins) {  // fewer than k tokens: nothing to cut
      z = mall;
      return true;
    }
    if (f.bucket == 0 || f.bucket == kValueSmall || f.bucket == kValueBins - 1) return false;
    const float pv = bin_value(f.bucket);
    u64 m = k - f.cnt_before;  // of the tokens equal to pv, the lowest-index m are kept
    const u64 w = units(pv);
    if (by_mass) m = (need - f.mass_before + w - 1) / w;
    z = f.mass_before + m * w;
    if (m < f.cnt_in) {
      u64 tot;
      auto tied = [&](float l, int i) { return (u64)(l == pv && (!some || kept(l, i)) ? 1 : 0); };
      auto which = [&](u64) { return m - 1; };
      const __nv_bfloat162 pv2 = __float2bfloat162_rn(pv), zero = __float2bfloat162_rn(0.f);
      cut = some ? search<T, kNT>(cl, sh, sl, rank, C, tied, which, &tot)
                 : search<T, kNT>(cl, sh, sl, rank, C, tied, which, &tot, [&](const uint4& r, int) {
                     __nv_bfloat162 w[4], c = zero;
                     memcpy(w, &r, sizeof(w));
#pragma unroll
                     for (int e = 0; e < 4; ++e) c = __hadd2(c, __heq2(w[e], pv2));  // 1 or 0
                     return (uint32_t)(__low2float(c) + __high2float(c));
                   });
    } else if (pv > pivot) {
      cut = 0x7fffffff;
    }
    pivot = pv;
    return true;
  };

  // The token of kept bf16 logits by their values' weights, after value_cut.
  auto value_search = [&]() {
    for (int b = 1 + tid; b < kValueBins - 1; b += kNT) {
      if (b == kValueSmall) continue;
      const float v = bin_value(b);
      sh.weight[bin_index(b)] = v >= pivot ? units(v) : 0;
    }
    __syncthreads();
    u64 tot;
    return search<T, kNT>(
        cl, sh, sl, rank, C, [&](float l, int i) { return kept(l, i) ? units(l) : 0ull; },
        [&](u64) { return mul_fraction(u, z, false); }, &tot,
        [&](const uint4& r, int i0) -> u64 {
          const uint32_t word[4] = {r.x, r.y, r.z, r.w};
          const float least = least_kept(i0);
          u64 t = 0;
          const bool mixed = least != least;  // the vector that holds the cut
          uint32_t odd = mixed ? 0xffu : 0u;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t c = value_index(word[e >> 1], e & 1);
            const float l = __uint_as_float(e & 1 ? word[e >> 1] & 0xffff0000u : word[e >> 1] << 16);
            const bool in = c < 2 * kValueOctaves;
            odd |= in || !(l >= kLowest) ? 0u : 1u << e;
            if (in && l >= least) t += sh.weight[c];
          }
#pragma unroll 1
          for (; odd; odd &= odd - 1) {  // as in value_cut
            const int i = i0 + __ffs(odd) - 1;
            const float l = sl.at(i);
            if (kept(l, i)) t += units(l);
          }
          return t;
        });
  };

  bool spread = false;   // the kept tokens are { kept }, spread over the CTAs
  bool exactly = false;  // no cheap way, or it was undecided
  if (temp == 0.f) {
    // greedy: the largest logit, lowest index
    int best = 0x7fffffff;
    if (tmax == mx) {
      float v[kN];
      sl.values(jmax, v);
#pragma unroll
      for (int e = kN - 1; e >= 0; --e)
        if (v[e] == mx) best = sl.first + jmax * kN + e;
    }
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) sh.warpi[warp] = best;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) best = min(best, sh.warpi[w]);
    publish(cl, sh.ccnt, rank, C, (uint32_t)best);
    cl.sync();
    for (int r = 0; r < C; ++r) best = min(best, (int)sh.ccnt[r]);
    pivot = mx;
    cut = best;
    token = best;
    z = 1ull << kOneBits;
  } else if ((by_maxima && (use_k || fast_ok)) || (use_m && !use_k)) {
    const FastScale fs(mx, chi, clo);
    const bool fast = !use_k && !use_m;  // top_p alone: its total is that of the whole row
    const float lo = fmaxf(pivot, guess);
    auto weights = [&](const uint4& r) {
      float v[kN];
      Vec<T>::unpack_clamped(r, fs.lmin, v);
      return __float2ull_rn(fs.template sum<kN, true>(v) * 17592186044416.f);
    };
    u64 z_fast;
    const int n = fast ? gather(lo, kSlots / C, all, weights, &z_fast)
                       : gather(lo, kSlots / C, all, nothing, &z_fast);
    // n tokens weigh at most n: too little for many a row that keeps more
    const bool enough = !fast || (u64)n << kOneBits >= share_of(top_p, z_fast);
    if (n <= kList && enough) listed = from_list(n, z_fast, fast);
    if (sizeof(T) == 4 && !listed && fast) {
      // A token outside the nucleus for sure: even V of its kind would hold less than 1 - top_p
      // of M's weight alone.  Tokens above that are counted per bucket.
      const float x0 = __log2f((1.f - top_p) / (float)V) - 0.02f;
      const float span = -x0 / chi;
      const float lx = fmaxf(mx - span - 1e-6f * (fabsf(mx) + span), kLowest);
      const float s2 = (float)(kBuckets - 1) / span;
      for (int i = tid; i < kBuckets; i += kNT) sh.hist[0][i] = 0;
      __syncthreads();
      sl.template each<2>([&](int, const uint4& r) {
        if (!(Vec<T>::largest(r) >= lx)) return;
        float v[kN];
        Vec<T>::unpack(r, v);
#pragma unroll
        for (int e = 0; e < kN; ++e)
          if (v[e] >= lx)
            atomicAdd(&sh.hist[0][__float2int_rz(fminf((mx - v[e]) * s2, (float)(kBuckets - 1)))], 1u);
      });
      const u64 need = share_of(top_p, z_fast);
      const u64 want = need + 2 * (need >> kRoughBits) + 2;
      // a token of bucket b weighs at least 2^(-(b + 1) / s2 chi), but the last also holds what
      // lies beyond its end
      const float per_bucket = -chi / s2;
      const Shared::Found f = join(
          false,
          [&](int b) {
            return b == kBuckets - 1
                       ? 0ull
                       : (u64)(17592186044416.f * 0.9999f * ex2f((float)(b + 1) * per_bucket));
          },
          0, [&](u64) { return want; });
      if (f.cnt_before + f.cnt_in <= (uint32_t)kList) {
        const float edge = mx - (float)(f.bucket + 1) / s2;
        const float low = fmaxf(lx, edge - 1e-6f * (fabsf(mx) + fabsf(edge)));
        u64 none;
        const int n2 = gather(low, kSlots / C, all, nothing, &none);
        if (n2 <= kList) listed = from_list(n2, z_fast, true);
      }
    }
    exactly = !listed;
  } else if (use_k || use_p) {
    exactly = true;
  } else {
    spread = true;
  }

  bool by_value = false;  // the last cut was one by values
  if (exactly) {
    // 1: cut by count (top-k, or no count cut at all when only min_p is set)
    if (use_k || use_m) {
      by_value = value_cut(false, use_k ? (uint32_t)top_k : 0x7fffffffu);
      if (!by_value) {
        histogram(false);
        const Shared::Found f =
            join(false, no_low, use_k ? (uint32_t)top_k : 0x7fffffffu, no_need);
        if (f.bucket < kBuckets) cut_bucket(f, false, (uint32_t)top_k - f.cnt_before, 0);
      }
    }
    // 2: cut by mass
    if (use_p) {
      by_value = value_cut(true, 0);
      if (!by_value) {
        histogram(true);
        const Shared::Found f = join(true, no_low, 0, [&](u64 t) { return share_of(top_p, t); });
        cut_bucket(f, true, 0, share_of(top_p, f.total) - f.mass_before);
      }
    }
    spread = true;
  }
  if (spread && pivot < INFINITY) {  // a pivot of kLowest too: it can hold the cut by index
    const int b = __float_as_int(pivot);
    above_pivot = pivot == 0.f ? __int_as_float(1) : __int_as_float(pivot > 0.f ? b + 1 : b - 1);
  }
  // some token above -inf is not kept
  const bool partial = pivot > kLowest || cut != 0x7fffffff;
  if (spread && by_value) {
    if constexpr (!kVerify) {
      // fast sums first where the smallest kept weight is well above their error
      u64 about;
      if (fast_ok && units(pivot) > z >> (kFastBits - 3))
        token = search_fast<T, kNT>(cl, sh, sl, rank, C, partial, kept,
                                    least_kept, FastScale(mx, chi, clo), units, u, &about);
      if (token < 0) token = value_search();
    }
  } else if (spread) {
    auto w_kept = [&](float l, int i) { return kept(l, i) ? units(l) : 0ull; };
    if constexpr (kVerify) {
      u64 s = 0;
      sl.template each<2>([&](int j, const uint4& r) {
        float v[kN];
        Vec<T>::unpack(r, v);
#pragma unroll
        for (int e = 0; e < kN; ++e) s += w_kept(v[e], sl.first + j * kN + e);
      });
      z = cluster_sum(s);
    } else {
      if (fast_ok)
        token = search_fast<T, kNT>(cl, sh, sl, rank, C, partial, kept,
                                    least_kept, FastScale(mx, chi, clo), units, u, &z);
      if (token < 0)
        token = search<T, kNT>(cl, sh, sl, rank, C, w_kept,
                          [&](u64 total) { return mul_fraction(u, total, false); }, &z);
    }
  }

  if constexpr (kVerify) {
    if (rank == 0 && tid == 0) {
      RowStats st;
      st.mx = mx;
      st.pivot = pivot;
      st.chi = chi;
      st.clo = clo;
      st.cut = cut;
      st.pad = 0;
      st.z = z;
      a.stats[row] = st;
      const int i = row % a.per;
      bool acc = false;
      if (i < a.gamma) {
        const int b = row / a.per;
        const int y = a.draft[(size_t)b * a.gamma + i];
        if (y < 0 || y >= V) {
          report(a.status, kStatusCheck, kKernSample);
        } else {
          const float l = to_f(lrow[y]);
          uint32_t mant;
          int n;
          // u q < w / Z, both sides times Z (w: units of 2^-44, 32 significant bits)
          if (kept(l, y) && weight_parts(l, mx, chi, clo, sh.tab, mant, n)) {
            const double w = __hiloint2double((n + kOneBits - 31 + 1023) << 20, 0) * (double)mant;
            acc = (double)u * (double)a.q[((size_t)b * a.gamma + i) * V + y] * (double)z < w;
          }
        }
      }
      a.accept[row] = acc ? 1 : 0;
    }
  } else {
    if (rank == 0 && tid == 0) a.tokens[row] = token;
    if (a.probs) {
      float* out = a.probs + (size_t)row * V;
      const float inv = __fdiv_rn(17592186044416.f, __ull2float_rn(z));  // 2^44 / Z
      auto exact_prob = [&](float l, float scale) {
        uint32_t mant;
        int n;
        if (!weight_parts(l, mx, chi, clo, sh.tab, mant, n)) return 0.f;
        // mant 2^-31 in [1, 2); 2^n in two factors, each a normal float
        const int h = n / 2;
        return (float)mant * (scale * 4.656612873e-10f) * __int_as_float((h + 127) << 23) *
               __int_as_float((n - h + 127) << 23);
      };
      if (listed) {
        if (rank == 0) {
          for (int i = tid; i < list_n; i += kNT) {
            const u64 k = sh.list.key[i];
            if (k > list_last) continue;
            out[(uint32_t)k] = exact_prob(key_value((uint32_t)(k >> 32)), inv);
          }
        }
      } else if (temp == 0.f) {
        fill_zero();
        __syncthreads();
        if (token >= sl.c0 && token < sl.c1 && tid == 0) out[token] = 1.f;
      } else {
        auto write = [&](int i0, const float* p) {
          if (i0 >= sl.c0 && i0 + kN <= sl.c1 && ((uintptr_t)(out + i0) & 15) == 0) {
#pragma unroll
            for (int e = 0; e < kN; e += 4)
              *reinterpret_cast<float4*>(out + i0 + e) =
                  make_float4(p[e], p[e + 1], p[e + 2], p[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < kN; ++e)
              if (i0 + e >= sl.c0 && i0 + e < sl.c1) out[i0 + e] = p[e];
          }
        };
        if (fast_ok) {
          const FastScale fs(mx, chi, clo);
          const u64 inv2 = pack2(inv, inv);
          sl.template each<2>([&](int j, const uint4& r) {
            float v[kN], p[kN];
            const int i0 = sl.first + j * kN;
            Vec<T>::unpack_clamped(r, fs.lmin, v);
#pragma unroll
            for (int e = 0; e < kN; e += 2)
              unpack2(mul2(fs.two(v[e], v[e + 1]), inv2), p[e], p[e + 1]);
            const float least = least_kept(i0);
            if (least == least) {
#pragma unroll
              for (int e = 0; e < kN; ++e) p[e] = v[e] >= least ? p[e] : 0.f;
            } else {
#pragma unroll
              for (int e = 0; e < kN; ++e)
                if (!kept(v[e], i0 + e)) p[e] = 0.f;
            }
            write(i0, p);
          });
        } else {
          sl.template each<1>([&](int j, const uint4& r) {
            float v[kN], p[kN];
            const int i0 = sl.first + j * kN;
            Vec<T>::unpack(r, v);
#pragma unroll
            for (int e = 0; e < kN; ++e) p[e] = kept(v[e], i0 + e) ? exact_prob(v[e], inv) : 0.f;
            write(i0, p);
          });
        }
      }
    }
  }
  // a CTA's shared memory stays valid until the others' last access: a listed row's is in
  // from_list or before
  if (!listed) cl.sync();
}

}  // namespace

template <typename T, bool kVerify, int kNT>
cudaError_t launch_filter_nt(const FilterArgs& a, long rows, cudaStream_t stream) {
  return launch_pdl_cluster(filter_kernel<T, kVerify, kNT>, dim3((unsigned)(rows * a.C)),
                            dim3(kNT), 0, stream, a.C, a);
}

}  // namespace dflash
