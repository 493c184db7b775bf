// Gradients of the attention of k_attn.hip from da, at the a and lse that it wrote:
//   p_ij = exp(s_ij - lse_i),  D_i = da_i . a_i
//   dv_j = sum_i p_ij da_i
//   ds_ij = p_ij (da_i . v_j - D_i), times 1 - tanh^2 with a cap
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
// Two kernels, each with the scores computed anew: one walks over the keys of 128
// queries (dq; it also writes lse in powers of two and D for the other), one over
// the queries of 128 keys and all the heads of their group (dk, dv).  Nothing is
// added from two sides: no atomics, sums in a fixed order.  That is 7 products
// where one walk with sums of dq in memory would have 5.
// p and ds are rounded to the inputs' type, as operands of products in that type.
#include "hna_internal.h"
#include "hna_attn.h"

namespace hna {
namespace {

using namespace attn;

// score in powers of two, and (CAP) the cap's slope, of a product x
template <typename T, bool CAP, bool BIAS>
__device__ inline float score(float x, float c1, float cap, float slope, float distance, float& bent) {
  x *= c1;
  if constexpr (CAP) {
    const float t = tanh_of<T>(x);
    bent = fmaf(-t, t, 1.0f);
    x = cap * t;
  }
  if constexpr (BIAS) x = fmaf(-slope, fabsf(distance), x);
  return x;
}

template <typename T, int DT, bool CAP, bool BIAS>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attn_dq_kernel(const AttnParams p) {
  typedef Tile<T, DT> L;
  __shared__ __attribute__((aligned(512))) unsigned char lds[4 * L::BYTES];   // K, V of two tiles
  __shared__ int span[4][2];
  __shared__ uint32_t bad[2], again;
  const int tid = threadIdx.x, l = tid & 63, up = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

  // blocks as in the forward pass
  const int nq = (int)((p.T + 127) / 128), r = p.H / p.G, total = nq * p.H;
  const int per_xcd = (total + 7) / 8, slot = (int)(blockIdx.x >> 3), n = (int)(blockIdx.x & 7) * per_xcd + slot;
  if (slot >= per_xcd || n >= total) return;
  const int gi = n / (nq * r), rem = n - gi * nq * r, qt = nq - 1 - rem / r;
  const int h = p.head_order[gi * r + rem % r], g = p.head_group[h];

  const int64_t q0 = (int64_t)qt * 128, t = q0 + 32 * w + (l & 31);
  const Span mine = Span::of(p.rows, p.causal, p.T, t);
  const int lo = mine.lo, hi = mine.hi;
  {
    // the keys that any query of the workgroup sees
    const bool on = mine.live && lo < hi;
    const int a = wave_min(on ? lo : INT32_MAX), b = wave_max(on ? hi : 0);
    if (l == 0) {
      span[w][0] = a;
      span[w][1] = b;
    }
    if (tid < 2) bad[tid] = 0;
    if (tid == 0) again = 0;
  }
  __syncthreads();
  const int first = __builtin_amdgcn_readfirstlane(min(min(span[0][0], span[1][0]), min(span[2][0], span[3][0])));
  const int end = __builtin_amdgcn_readfirstlane(max(max(span[0][1], span[1][1]), max(span[2][1], span[3][1])));

  const T* K = static_cast<const T*>(p.k) + (int64_t)g * p.d;
  const T* V = static_cast<const T*>(p.v) + (int64_t)g * p.d;
  uint32_t ko[L::PERIOD], vo[L::PERIOD];
  L::offsets(ko, w, l, p.ld_k, p.d);
  L::offsets(vo, w, l, p.ld_v, p.d);
  const uint32_t base = lds_addr(lds);
  const typename L::At lane0 = L::lane(base, l);
  auto issue = [&](int kb, int buf) __attribute__((always_inline)) {
    L::copy(K, p.ld_k, p.d, kb, end, ko, base + (uint32_t)(buf * 2 * L::BYTES), w);
    L::copy(V, p.ld_v, p.d, kb, end, vo, base + (uint32_t)(buf * 2 * L::BYTES + L::BYTES), w);
  };

  typename L::Frag qf[2 * DT], af[2 * DT];
  const int64_t tr = min<int64_t>(t, p.T - 1);
  const T* qrow = static_cast<const T*>(p.q) + tr * p.ld_q + (int64_t)h * p.d;
  const T* darow = static_cast<const T*>(p.da) + (tr * p.H + h) * p.d;
  const T* arow = static_cast<const T*>(p.a) + (tr * p.H + h) * p.d;
  float D = 0.f;
#pragma unroll
  for (int s = 0; s < 2 * DT; ++s) {
    L::load(qf[s], qrow, s, p.d, l);
    L::load(af[s], darow, s, p.d, l);
    typename L::Frag y;
    L::load(y, arow, s, p.d, l);
    constexpr int N = 8;
    T x[N], z[N];
    __builtin_memcpy(x, af[s], sizeof(x));
    __builtin_memcpy(z, y, sizeof(z));
#pragma unroll
    for (int e = 0; e < N; ++e) D = fmaf((float)x[e], (float)z[e], D);
  }
  D = swap_sum(D);
  const float lse = p.lse[tr * p.H + h];
  const float lse2 = lse == -__builtin_inff() ? __builtin_inff() : kLog2e * lse;   // a row that sees nothing: p = 0
  if (up == 0 && t < p.T) {
    p.stat[(int64_t)h * p.T + t] = lse2;
    p.stat[((int64_t)p.H + h) * p.T + t] = D;
  }

  f32x16 o[DT];
  const float c1 = CAP ? 2.0f * kLog2e * p.scale / p.cap : kLog2e * p.scale;
  const float cap = kLog2e * p.cap;
  const float slope = BIAS ? kLog2e * p.slopes[h] : 0.f;

  // the walk over the keys, as in the forward pass: again and CAREFUL with the keys
  // where a sum is not finite
  auto walk = [&](auto careful) __attribute__((always_inline)) {
    constexpr bool CAREFUL = decltype(careful)::value;
    int buf = 0;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = f32x16{};
    if (first < end) issue(first, 0);
    for (int kb = first; kb < end; kb += 64, buf ^= 1) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (kb + 64 < end) issue(kb + 64, buf ^ 1);
      const typename L::At kt = L::move(lane0, (uint32_t)(buf * 2 * L::BYTES)), vt = L::move(kt, L::BYTES);
      uint32_t bad0 = 0, bad1 = 0;
      if constexpr (CAREFUL) {
        L::find_bad(lds + buf * 2 * L::BYTES, tid, 256, bad);
        __syncthreads();
        bad0 = __builtin_amdgcn_readfirstlane(bad[0]);
        bad1 = __builtin_amdgcn_readfirstlane(bad[1]);
        __syncthreads();
        if (tid < 2) bad[tid] = 0;
      }
      if (!__any(mine.live && lo < kb + 64 && hi > kb)) continue;
      const bool whole = __all(!mine.live || (lo <= kb && hi >= kb + 64));
      const float at = (float)((int)t - kb - 4 * up);
      const uint32_t from = (uint32_t)(lo - kb - 4 * up), len = (uint32_t)max(hi - lo, 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f32x16 s = {}, dp = {};
#pragma unroll
        for (int x = 0; x < 2 * DT; ++x) {
          typename L::Frag a;
          L::rows(a, kt, 32 * i, x);
          mma(s, a, qf[x]);
          L::rows(a, vt, 32 * i, x);
          mma(dp, a, af[x]);
        }
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int off = 32 * i + 8 * (v >> 2) + (v & 3);
          float bent = 1.f;
          const float y = score<T, CAP, BIAS>(s[v], c1, cap, slope, at - (float)off, bent);
          float ds = __builtin_amdgcn_exp2f(y - lse2) * (dp[v] - D);
          if constexpr (CAP) ds *= bent;
          s[v] = ds;
        }
        if (!whole) {
#pragma unroll
          for (int v = 0; v < 16; ++v) s[v] = (uint32_t)(32 * i + 8 * (v >> 2) + (v & 3)) - from < len ? s[v] : 0.f;
        }
        L::template along<CAREFUL>(o, kt, 32 * i, s, l);
        if constexpr (CAREFUL)
          add_bad_rows<T, DT>(o, s, i ? bad1 : bad0, p.d, l, [&](int x) { return K + (int64_t)(kb + 32 * i + x) * p.ld_k; },
                              [&](int x) { return kb + 32 * i + x >= lo && kb + 32 * i + x < hi; });
      }
    }
  };
  walk(std::false_type{});
  const float z = finite<DT>(o);
  if (__any(mine.live && z != z)) again = 1;
  __syncthreads();
  if (again) walk(std::true_type{});
  if (!mine.live) return;
  T* out = static_cast<T*>(p.dq) + (t * p.H + h) * p.d;
  const float sc = p.scale;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int e = 32 * i + 8 * a + 4 * up;
      if (e < p.d)
        *reinterpret_cast<typename Four<T>::type*>(out + e) = Four<T>::of(o[i][4 * a] * sc, o[i][4 * a + 1] * sc, o[i][4 * a + 2] * sc, o[i][4 * a + 3] * sc);
    }
}

// A workgroup has 128 keys of a group, 32 a wave, and walks over tiles of 64 queries
// of each of the group's heads; a lane holds one key.  bf16: 8 waves, of which two
// share keys and take 32 queries of a tile each (their sums meet in LDS at the end),
// and v's rows are read from LDS: dk, dv and k's rows leave no registers for them at
// two waves a SIMD.  fp32: 4 waves, all of it in registers at one wave a SIMD.
template <typename T, int DT, bool CAP, bool BIAS>
__global__ __launch_bounds__(sizeof(T) == 2 ? 512 : 256) void attn_dkv_kernel(const AttnParams p) {
  typedef Tile<T, DT> L;
  constexpr bool SPLIT = sizeof(T) == 2;
  constexpr int NW = SPLIT ? 8 : 4;
  __shared__ __attribute__((aligned(512))) unsigned char lds[(SPLIT ? 6 : 4) * L::BYTES];   // Q, dA of two tiles; V
  __shared__ __attribute__((aligned(16))) float stat[2][2][64];              // lse2, D
  __shared__ __attribute__((aligned(16))) int4 sees[2][64];
  __shared__ __attribute__((aligned(16))) uint32_t seen[NW][64];             // of a wave's keys, by query
  __shared__ int span[4][2];
  __shared__ uint32_t bad[4], again;                                         // of Q, of dA
  const int tid = threadIdx.x, l = tid & 63, up = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = w & 3, half = w >> 2;                        // keys; (SPLIT) queries of a tile

  // blocks of an XCD are consecutive: the keys from the first on (with the longest columns), then the groups
  const int nk = (int)((p.T + 127) / 128), total = nk * p.G;
  const int per_xcd = (total + 7) / 8, slot = (int)(blockIdx.x >> 3), n = (int)(blockIdx.x & 7) * per_xcd + slot;
  if (slot >= per_xcd || n >= total) return;
  const int g = n / nk, k0 = (n - g * nk) * 128;
  const int heads0 = p.group_start[g], heads = p.group_start[g + 1] - heads0;

  const int64_t t = (int64_t)k0 + 32 * wk + (l & 31);
  bool live = t < p.T;
  int qfirst = 0, qend = 0;                                   // the queries that see this lane's key
  if (live) {
    if (p.rows) {
      const int4 v = p.rows[t];
      live = v.x >= 0;
      qfirst = max(v.z, 0);
      qend = live ? (int)min<int64_t>(max(v.w, 0), p.T) : 0;
    } else {
      qfirst = p.causal ? (int)t : 0;
      qend = (int)p.T;
    }
  }
  {
    const bool on = qfirst < qend;
    const int a = wave_min(on ? qfirst : INT32_MAX), b = wave_max(on ? qend : 0);
    if (l == 0 && half == 0) {
      span[wk][0] = a;
      span[wk][1] = b;
    }
    if (tid < 4) bad[tid] = 0;
    if (tid == 0) again = 0;
  }
  __syncthreads();
  const int first = __builtin_amdgcn_readfirstlane(min(min(span[0][0], span[1][0]), min(span[2][0], span[3][0])));
  const int end = __builtin_amdgcn_readfirstlane(max(max(span[0][1], span[1][1]), max(span[2][1], span[3][1])));
  const int tiles = first < end ? (end - first + 63) / 64 : 0, steps = tiles * heads;

  const int64_t ld_a = (int64_t)p.H * p.d;
  const uint32_t base = lds_addr(lds);
  const typename L::At lane0 = L::lane(base, l);
  uint32_t qo[L::PERIOD], ao[L::PERIOD];                      // SPLIT: waves 0 .. 3 copy Q, 4 .. 7 dA
  L::offsets(qo, wk, l, SPLIT && half ? ld_a : p.ld_q, p.d);
  if constexpr (!SPLIT) L::offsets(ao, wk, l, ld_a, p.d);
  int ih = 0, it = 0;                                         // the copies' head and tile
  auto issue = [&](int buf) __attribute__((always_inline)) {
    const int h = p.head_order[heads0 + ih], qb = first + 64 * it;
    const T* q = static_cast<const T*>(p.q) + (int64_t)h * p.d;
    const T* da = static_cast<const T*>(p.da) + (int64_t)h * p.d;
    const uint32_t to = base + (uint32_t)(buf * 2 * L::BYTES);
    if constexpr (SPLIT) {
      L::copy(half ? da : q, half ? ld_a : p.ld_q, p.d, qb, end, qo, to + (uint32_t)(half * L::BYTES), wk);
    } else {
      L::copy(q, p.ld_q, p.d, qb, end, qo, to, wk);
      L::copy(da, ld_a, p.d, qb, end, ao, to + L::BYTES, wk);
    }
    const uint32_t left = (uint32_t)min(end - qb, 64);
    if (w < 2) dma4s(uniform_rsrc(p.stat + ((int64_t)w * p.H + h) * p.T + qb, 4 * left), 4u * (uint32_t)l, lds_addr(stat[buf][w]));
    if (w == 2 && p.rows) dma16s(uniform_rsrc(p.rows + qb, 16 * left), 16u * (uint32_t)l, 0u, lds_addr(sees[buf]));
    if (++it == tiles) {
      it = 0;
      ++ih;
    }
  };

  const int64_t tr = min<int64_t>(t, p.T - 1);
  typename L::Frag kf[2 * DT], vf[SPLIT ? 1 : 2 * DT];
  const T* krow = static_cast<const T*>(p.k) + tr * p.ld_k + (int64_t)g * p.d;
#pragma unroll
  for (int s = 0; s < 2 * DT; ++s) L::load(kf[s], krow, s, p.d, l);
  if constexpr (SPLIT) {
    uint32_t vo[L::PERIOD];
    L::offsets(vo, wk, l, p.ld_v, p.d);
    L::copy(static_cast<const T*>(p.v) + (int64_t)g * p.d, p.ld_v, p.d, k0 + 64 * half, p.T, vo, base + (uint32_t)((4 + half) * L::BYTES), wk);
  } else {
    const T* vrow = static_cast<const T*>(p.v) + tr * p.ld_v + (int64_t)g * p.d;
#pragma unroll
    for (int s = 0; s < 2 * DT; ++s) L::load(vf[s], vrow, s, p.d, l);
  }
  const typename L::At vt = L::move(lane0, (uint32_t)((4 + (wk >> 1)) * L::BYTES + (wk & 1) * 32 * L::PITCH));

  f32x16 dk[DT], dv[DT];
  const float c1 = CAP ? 2.0f * kLog2e * p.scale / p.cap : kLog2e * p.scale;
  const float cap = kLog2e * p.cap;
  const int kw = k0 + 32 * wk, kw_end = (int)min<int64_t>(kw + 32, p.T);

  // the walk over the queries, as in the forward pass: again and CAREFUL with q and
  // da where a sum is not finite
  auto walk = [&](auto careful) __attribute__((always_inline)) {
    constexpr bool CAREFUL = decltype(careful)::value;
    int buf = 0, head = 0, tile = 0;
    ih = it = 0;
#pragma unroll
    for (int i = 0; i < DT; ++i) dk[i] = dv[i] = f32x16{};
    if (steps > 0) issue(0);
    for (int step = 0; step < steps; ++step, buf ^= 1) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (step + 1 < steps) issue(buf ^ 1);
      const int h = p.head_order[heads0 + head], qb = first + 64 * tile;
      if (++tile == tiles) {
        tile = 0;
        ++head;
      }
      const float slope = BIAS ? kLog2e * p.slopes[h] : 0.f;
      const typename L::At qt = L::move(lane0, (uint32_t)(buf * 2 * L::BYTES)), at = L::move(qt, L::BYTES);
      uint32_t bad_q[2] = {0, 0}, bad_a[2] = {0, 0};
      if constexpr (CAREFUL) {
        L::find_bad(lds + buf * 2 * L::BYTES, tid, 64 * NW, bad);
        L::find_bad(lds + buf * 2 * L::BYTES + L::BYTES, tid, 64 * NW, bad + 2);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          bad_q[i] = __builtin_amdgcn_readfirstlane(bad[i]);
          bad_a[i] = __builtin_amdgcn_readfirstlane(bad[2 + i]);
        }
        __syncthreads();
        if (tid < 4) bad[tid] = 0;
      }
      // what query l of the tile sees: its keys [x, y)
      int2 sq;
      if (p.rows) {
        sq = *reinterpret_cast<const int2*>(&sees[buf][l]);      // zeros behind the last query
        if (sq.x < 0) sq.y = 0;
      } else {
        sq = make_int2(0, qb + l < p.T ? (p.causal ? qb + l + 1 : (int)p.T) : 0);
      }
      const bool mine = !SPLIT || up == half;
      if (!__any(mine && sq.x < kw_end && sq.y > kw)) continue;
      const bool whole = __all(!mine || (sq.x <= kw && sq.y >= kw_end));
      if (!whole || CAREFUL) {
        const uint32_t a = (uint32_t)min(max(sq.x - kw, 0), 32), b = (uint32_t)min(max(sq.y - kw, 0), 32);
        seen[w][l] = (uint32_t)((1ull << b) - 1) & ~(uint32_t)((1ull << a) - 1);
      }
      const float from = (float)((int)t - qb - 4 * up);
      auto block = [&](int i) __attribute__((always_inline)) {     // queries 32 i .. of the tile
        f32x16 s = {}, dp = {};
#pragma unroll
        for (int x = 0; x < 2 * DT; ++x) {
          typename L::Frag a, b;
          L::rows(a, qt, 32 * i, x);
          mma(s, a, kf[x]);
          L::rows(a, at, 32 * i, x);
          if constexpr (SPLIT) {
            L::rows(b, vt, 0, x);
            mma(dp, a, b);
          } else {
            mma(dp, a, vf[x]);
          }
        }
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int q = 32 * i + 8 * a + 4 * up;
          const float4 l4 = *reinterpret_cast<const float4*>(&stat[buf][0][q]), d4 = *reinterpret_cast<const float4*>(&stat[buf][1][q]);
          const float ls[4] = {l4.x, l4.y, l4.z, l4.w}, D[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int v = 4 * a + e;
            float bent = 1.f;
            const float y = score<T, CAP, BIAS>(s[v], c1, cap, slope, from - (float)(32 * i + 8 * a + e), bent);
            const float pr = __builtin_amdgcn_exp2f(y - ls[e]);
            float ds = pr * (dp[v] - D[e]);
            if constexpr (CAP) ds *= bent;
            dp[v] = pr;
            s[v] = ds;
          }
        }
        if (!whole) {
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const uint4 m4 = *reinterpret_cast<const uint4*>(&seen[w][32 * i + 8 * a + 4 * up]);
            const uint32_t m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool on = (m[e] >> (l & 31)) & 1;
              dp[4 * a + e] = on ? dp[4 * a + e] : 0.f;
              s[4 * a + e] = on ? s[4 * a + e] : 0.f;
            }
          }
        }
        L::template along<CAREFUL>(dv, at, 32 * i, dp, l);
        L::template along<CAREFUL>(dk, qt, 32 * i, s, l);
        if constexpr (CAREFUL) {
          auto on = [&](int x) { return ((seen[w][32 * i + x] >> (l & 31)) & 1) != 0; };
          add_bad_rows<T, DT>(dv, dp, i ? bad_a[1] : bad_a[0], p.d, l, [&](int x) { return static_cast<const T*>(p.da) + (int64_t)(qb + 32 * i + x) * ld_a + (int64_t)h * p.d; }, on);
          add_bad_rows<T, DT>(dk, s, i ? bad_q[1] : bad_q[0], p.d, l, [&](int x) { return static_cast<const T*>(p.q) + (int64_t)(qb + 32 * i + x) * p.ld_q + (int64_t)h * p.d; }, on);
        }
      };
      if constexpr (SPLIT) {
        block(half);
      } else {
        block(0);
        block(1);
      }
    }
  };
  walk(std::false_type{});
  const float z = finite<DT>(dk) + finite<DT>(dv);
  if (__any(live && z != z)) again = 1;
  __syncthreads();
  if (again) walk(std::true_type{});

  const float sc = p.scale;
  auto put = [&](f32x16 (&x)[DT], void* to, float by) __attribute__((always_inline)) {
    if constexpr (SPLIT) {
      // the second half's sums to the first, through the stages
      constexpr int OP = 32 * DT + 4;
      static_assert(4 * 32 * OP * 4 <= 6 * L::BYTES, "the sums of four waves fit");
      float* o = reinterpret_cast<float*>(lds) + (wk * 32 + (l & 31)) * OP;
      __syncthreads();
      if (half) {
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int a = 0; a < 4; ++a)
            *reinterpret_cast<float4*>(o + 32 * i + 8 * a + 4 * up) = make_float4(x[i][4 * a], x[i][4 * a + 1], x[i][4 * a + 2], x[i][4 * a + 3]);
      }
      __syncthreads();
      if (half) return;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const float4 v = *reinterpret_cast<const float4*>(o + 32 * i + 8 * a + 4 * up);
          x[i][4 * a] += v.x;
          x[i][4 * a + 1] += v.y;
          x[i][4 * a + 2] += v.z;
          x[i][4 * a + 3] += v.w;
        }
    }
    if (!live) return;
    T* out = static_cast<T*>(to) + (t * p.G + g) * p.d;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int e = 32 * i + 8 * a + 4 * up;
        if (e < p.d) *reinterpret_cast<typename Four<T>::type*>(out + e) = Four<T>::of(x[i][4 * a] * by, x[i][4 * a + 1] * by, x[i][4 * a + 2] * by, x[i][4 * a + 3] * by);
      }
  };
  put(dk, p.dk, sc);
  put(dv, p.dv, 1.f);
}

template <typename T, int DT, bool CAP, bool BIAS>
hipError_t launch_one(const AttnParams& p, hipStream_t st) {
  const int64_t blocks = (p.T + 127) / 128, nq = blocks * p.H, nk = blocks * p.G;
  hipLaunchKernelGGL((attn_dq_kernel<T, DT, CAP, BIAS>), dim3((unsigned)(8 * ((nq + 7) / 8))), dim3(256), 0, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_dkv_kernel<T, DT, CAP, BIAS>), dim3((unsigned)(8 * ((nk + 7) / 8))), dim3(sizeof(T) == 2 ? 512 : 256), 0, st, p);
  return hipGetLastError();
}
template <typename T, int DT>
hipError_t launch_dt(const AttnParams& p, hipStream_t st) {
  if (p.cap > 0.f) return p.slopes ? launch_one<T, DT, true, true>(p, st) : launch_one<T, DT, true, false>(p, st);
  return p.slopes ? launch_one<T, DT, false, true>(p, st) : launch_one<T, DT, false, false>(p, st);
}
template <typename T>
hipError_t launch_t(const AttnParams& p, hipStream_t st) {
  if (p.d <= 32) return launch_dt<T, 1>(p, st);
  if (p.d <= 64) return launch_dt<T, 2>(p, st);
  if (p.d <= 96) return launch_dt<T, 3>(p, st);
  return launch_dt<T, 4>(p, st);
}

}  // namespace

hipError_t launch_attention_backward(const AttnParams& p, int bf16, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  return bf16 ? launch_t<__bf16>(p, st) : launch_t<float>(p, st);
}

}  // namespace hna
