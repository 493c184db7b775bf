// 8-bit integer product on the matrix cores:
//   out[t, n] = (sum_k q[t, k] w[n, k]) q_scale[t] w_scale[n]
// for one weight matrix or two of one shape (an FFN's gate and up) in one launch;
// q [T, K] and w [N, K] row-major with k contiguous, sums in int32 (exact for
// K < 2^17), the scales applied in fp32, one rounding to the output type.
// The channels are the MFMA rows and the tokens its columns, so a lane ends up
// with 4 consecutive channels of one token: out's contiguous direction.
// Three kernels: 256 x 256 tiles for large products, smaller tiles where those
// would leave CUs idle, and no tiles at all for a few tokens.  The borders are
// in launch_mm_int.
#include "hna_internal.h"
#include "hna_hot.h"

namespace hna {
namespace {

using namespace hot;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

__device__ inline void mma_int(i32x16& c, const uint4& a, const uint4& b) {
  c = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// 4 consecutive channels n .. n + 3 of token t
__device__ inline void put4(const IntMmParams& p, int z, int64_t t, int n, const int (&v)[4], float st) {
  const float* w_scale = z ? p.w_scale[1] : p.w_scale[0];
  void* out = z ? p.out[1] : p.out[0];
  const int64_t o = t * p.N + n;
  if (n + 4 <= p.N && p.N % 4 == 0) {
    const float4 sw = *reinterpret_cast<const float4*>(w_scale + n);
    const float f[4] = {(float)v[0] * st * sw.x, (float)v[1] * st * sw.y, (float)v[2] * st * sw.z, (float)v[3] * st * sw.w};
    if (p.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(out) + o) = make_float4(f[0], f[1], f[2], f[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p.N) break;
    const float f = (float)v[e] * st * w_scale[n + e];
    if (p.out_bf16) static_cast<uint16_t*>(out)[o + e] = (uint16_t)pack_bf16x2(f, 0.f);
    else static_cast<float*>(out)[o + e] = f;
  }
}

// Tiles of BM x BN: KG groups of WGM x WGN waves, each group with a part of k of
// its own (128 bytes of a step of KG 128), the steps in a ring of NST stages.
// Several groups shorten the chain of steps where there are few tiles: a step
// takes about 0.26 us however little it computes (a barrier, then LDS reads,
// then the MFMAs that wait for them).  The groups' sums meet in LDS.
// 16 to 2000 tokens x 14336 x 4096, weights read from HBM: 18 to 122 us, 1.3
// to 3.5 times the larger of the bytes at 6.0 TB/s and the operations at 2.57e15.
template <int BM, int BN, int WGM, int WGN, int KG, int NST>
__global__ __launch_bounds__(64 * WGM * WGN * KG) void mm_int_kernel(const IntMmParams p) {
  constexpr int NW = WGM * WGN, NT = 64 * NW * KG;
  constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  constexpr int ROWS = BM + BN, BK = 128, CPR = BK / 16, RPI = 64 / CPR;
  constexpr int PART = ROWS * BK, STAGE = KG * PART;
  constexpr int NCP = ROWS / (RPI * NW), NCX = BM / (RPI * NW);
  constexpr int PITCH = BM + 4;                          // ints of a token's row of sums
  static_assert(BM % (RPI * NW) == 0 && BN % (RPI * NW) == 0, "copy rounds cover whole rows");
  static_assert((NST - 2) * NCP <= 63, "copies in flight must fit the wait counter");
  constexpr int SUMS = BN * PITCH * 4;
  __shared__ __attribute__((aligned(16))) unsigned char lds[NST * STAGE > SUMS ? NST * STAGE : SUMS];

  const int tid = threadIdx.x, l = tid & 63;
  const int wg = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wg / NW, w = wg % NW;
  const int wm = w / WGN, wn = w % WGN;

  const int z = blockIdx.y;
  const float* w_scale = z ? p.w_scale[1] : p.w_scale[0];
  void* out = z ? p.out[1] : p.out[0];

  // tile of this workgroup: XCD by XCD, in groups of 4 tile rows
  const int ntm = (p.N + BM - 1) / BM;
  const int64_t ntn = (p.T + BN - 1) / BN, ntiles = ntm * ntn;
  const int64_t per_xcd = (ntiles + 7) / 8;
  const int64_t t = (int64_t)(blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per_xcd || t >= ntiles) return;
  constexpr int GM = 4;
  const int64_t gsize = GM * ntn;
  const int g0 = (int)(t / gsize) * GM, gm = min(GM, ntm - g0);
  const int64_t tg = t - (t / gsize) * gsize;
  const int n0 = (g0 + (int)(tg % gm)) * BM;
  const int64_t t0 = tg / gm * BN;

  const int64_t xb = (int64_t)(p.N - n0) * p.K, yb = (p.T - t0) * p.K;
  const u32x4 rx = uniform_rsrc((z ? p.w[1] : p.w[0]) + (int64_t)n0 * p.K, xb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)xb);
  const u32x4 ry = uniform_rsrc(p.q + t0 * p.K, yb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)yb);

  i32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x16{};
  const int nk = (p.K + KG * BK - 1) / (KG * BK);

  // copy i of wave w fills rows RPI (NW i + w) .. + RPI - 1 of its group's part
  // (w rows first); rows past the end and bytes past K read zeros
  uint32_t voff[NCP];
  int kc[NCP];
#pragma unroll
  for (int i = 0; i < NCP; ++i) {
    const int r = RPI * (NW * i + w) + l / CPR;
    kc[i] = grp * BK + 16 * ((l % CPR) ^ swz<CPR>(r));
    voff[i] = (uint32_t)((int64_t)(i < NCX ? r : r - BM) * p.K + kc[i]);
  }
  const uint32_t lds0 = lds_addr(lds) + (uint32_t)(grp * PART + w * 1024);
  auto issue = [&](int k0, int buf) __attribute__((always_inline)) {
    const uint32_t base = lds0 + (uint32_t)(buf * STAGE);
    const uint32_t soff = __builtin_amdgcn_readfirstlane((uint32_t)k0);
#pragma unroll
    for (int i = 0; i < NCP; ++i)
      dma16s(i < NCX ? rx : ry, k0 + kc[i] >= p.K ? kOutOfRange : voff[i], soff, base + (uint32_t)(i * NW * 1024));
  };

#pragma unroll
  for (int st = 0; st < NST - 1; ++st) issue(st * KG * BK, st);
  int cur = 0;
  for (int kt = 0; kt < nk; ++kt) {
    // step kt has landed once at most the copies of the NST - 2 steps after it
    // are in flight (past k they read zeros); the barrier shows it to every wave
    // and ends their reads of step kt - 1, whose stage the next copies take
    __builtin_amdgcn_s_waitcnt(vm_wait((NST - 2) * NCP));
    __syncthreads();
    issue((kt + NST - 1) * KG * BK, cur == 0 ? NST - 1 : cur - 1);
    const unsigned char* sb = lds + cur * STAGE + grp * PART;
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks) {
      const int col = 2 * ks + (l >> 5);
      uint4 fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = wm * WM + i * 32 + (l & 31);
        fa[i] = *reinterpret_cast<const uint4*>(sb + r * BK + ((col ^ swz<CPR>(r)) << 4));
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int r = BM + wn * WN + j * 32 + (l & 31);
        fb[j] = *reinterpret_cast<const uint4*>(sb + r * BK + ((col ^ swz<CPR>(r)) << 4));
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) mma_int(acc[i][j], fa[i], fb[j]);
    }
    cur = cur + 1 == NST ? 0 : cur + 1;
  }

  // the sums as rows of a token's BM channels, in the stages: lane l holds token
  // (l & 31) and channels 8 a + 4 (l / 32) + e of each 32 x 32 tile
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // the last copies (zeros) are in
  __syncthreads();
  int* sums = reinterpret_cast<int*>(lds);
#pragma unroll
  for (int x = 0; x < KG; ++x) {
    if (grp == x) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            int4* d = reinterpret_cast<int4*>(sums + (wn * WN + j * 32 + (l & 31)) * PITCH + wm * WM + i * 32 + 8 * a + 4 * (l >> 5));
            int4 v = make_int4(acc[i][j][4 * a], acc[i][j][4 * a + 1], acc[i][j][4 * a + 2], acc[i][j][4 * a + 3]);
            if (x > 0) {
              const int4 o = *d;
              v = make_int4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
            }
            *d = v;
          }
    }
    __syncthreads();
  }
  const int rows = (int)min<int64_t>(BN, p.T - t0);
  if (p.N % 8 == 0) {
    for (int x = tid * 8; x < BM * BN; x += NT * 8) {
      const int r = x / BM, c = x % BM, n = n0 + c;
      if (r >= rows || n >= p.N) continue;
      const int4 a = *reinterpret_cast<const int4*>(sums + r * PITCH + c), b = *reinterpret_cast<const int4*>(sums + r * PITCH + c + 4);
      const float4 s = *reinterpret_cast<const float4*>(w_scale + n), u = *reinterpret_cast<const float4*>(w_scale + n + 4);
      const float st = p.q_scale[t0 + r];
      const int64_t o = (t0 + r) * p.N + n;
      const float4 v = make_float4((float)a.x * st * s.x, (float)a.y * st * s.y, (float)a.z * st * s.z, (float)a.w * st * s.w);
      const float4 y = make_float4((float)b.x * st * u.x, (float)b.y * st * u.y, (float)b.z * st * u.z, (float)b.w * st * u.w);
      if (p.out_bf16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o) =
            make_uint4(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      } else {
        reinterpret_cast<float4*>(static_cast<float*>(out) + o)[0] = v;
        reinterpret_cast<float4*>(static_cast<float*>(out) + o)[1] = y;
      }
    }
  } else if (!p.out_bf16) {
    for (int x = tid; x < BM * BN; x += NT) {
      const int r = x / BM, c = x % BM, n = n0 + c;
      if (r >= rows || n >= p.N) continue;
      static_cast<float*>(out)[(t0 + r) * p.N + n] = (float)sums[r * PITCH + c] * p.q_scale[t0 + r] * w_scale[n];
    }
  } else {
    // rows that start on any element: pairs that lie on 4 bytes, and the elements left at both ends
    uint16_t* o = static_cast<uint16_t*>(out);
    const int m = min(BM, p.N - n0);
    auto value = [&](int r, int c) { return (float)sums[r * PITCH + c] * p.q_scale[t0 + r] * w_scale[n0 + c]; };
    for (int x = tid; x < BM / 2 * BN; x += NT) {
      const int r = x / (BM / 2), odd = (int)((t0 + r) & p.N & 1), c = 2 * (x % (BM / 2)) + odd;
      if (r >= rows || c + 1 >= m) continue;
      *reinterpret_cast<uint32_t*>(o + (t0 + r) * p.N + n0 + c) = pack_bf16x2(value(r, c), value(r, c + 1));
    }
    for (int x = tid; x < 2 * BN; x += NT) {
      const int r = x >> 1, odd = (int)((t0 + r) & p.N & 1), c = x & 1 ? m - 1 : 0;
      if (r < rows && (x & 1 ? (m - odd) & 1 : odd))
        o[(t0 + r) * p.N + n0 + c] = (uint16_t)pack_bf16x2(value(r, c), 0.f);
    }
  }
}

// Large products: 256 x 256 tiles on 4 waves, one per SIMD, each 128 x 128 (16
// accumulators of 32 x 32: the largest wave tile, so that fragment reads and
// copies together keep LDS busy 3/4 of the MFMA time).  128 bytes of k a step
// (whole cache lines) in two stages.  A step is four quarters of 32 bytes; the
// fragments of the next quarter are read while the MFMAs of this one run:
//   quarters 0 .. 2 of step g, reading quarters 1 .. 3
//   wait for the reads and for step g + 1's copies; barrier
//   quarter 3, reading quarter 0 of step g + 1 and copying step g + 2 over step g
// The barrier says that every wave holds step g in registers (its stage is
// free) and that every wave's part of step g + 1 is in LDS.
// One workgroup a CU walks over its tiles, and the steps of all of them are one
// stream: the last two steps of a tile copy the first two of the next, so the
// copies never drain, and the output's stores overlap the next tile's MFMAs.
// Copies have one step (about 1 us) to arrive, which the L2 keeps to and HBM
// does not: a third stream touches the lines of step g + 3 (a fifth faster on
// zeros, 3% on data, where power sets the pace), each workgroup of
// an XCD its share of the panels it has in common with its neighbours.
// (The scales of a tile come with its first step, into the half of their
// buffer that the tile before the last one had: a tile has two steps at least.)
// Measured (operations a second), T x K x N: 16384 x 14336 x 4096 0.73 to 0.75
// ms, 2.6e15, MFMAs busy 70% of the cycles at 1.76 GHz: the clock that power
// leaves (an earlier form: 2.25e15, on zeros 3.4e15).  65536 x 1536 x 4096 0.40 to
// 0.41 ms, 2.0e15: 5.5 us of a tile's 25.6 pass outside its steps (from K 1024,
// 2048 and 4096).  The first dozen calls after an idle time take up to 0.87 and
// 0.53 ms.  An int32 library product, settled: 0.719 ms, 2.68e15, against 0.742
// here in the same run, and 0.477 ms, 1.7e15, against 0.40.
// Every wait counts operations in flight, so a step issues the same number of
// them everywhere: reads past the end of an operand return zeros and stores
// past the end of out are dropped by the buffer's range.
struct IntTiles {
  int ntm1, ntm, gsize, ntiles, last, slots;
};
// where a tile lies, and its operands from its first row on
struct IntPanels {
  u32x4 w, q;
  int z, n0, ni, ti;   // matrix, first channel; position in its group of 4 x (tokens) tiles
  __device__ inline void set(const IntMmParams& p, const IntTiles& g, int t) {
    const int grp = t / g.gsize, tg = t - grp * g.gsize;
    const int gm = min(4, g.ntm - grp * 4);
    ti = tg / max(gm, 1);
    ni = tg - ti * gm;
    const int tn = grp * 4 + ni;                          // both matrices' tiles in a row
    z = tn >= g.ntm1 ? 1 : 0;
    n0 = (tn - z * g.ntm1) * 256;
    const bool none = t >= g.ntiles;
    const int64_t t0 = (int64_t)ti * 256;
    const int64_t xb = none ? 0 : (int64_t)(p.N - n0) * p.K, yb = none ? 0 : (p.T - t0) * p.K;
    w = uniform_rsrc((z ? p.w[1] : p.w[0]) + (none ? 0 : (int64_t)n0 * p.K), xb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)xb);
    q = uniform_rsrc(p.q + (none ? 0 : t0 * p.K), yb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)yb);
  }
};

// The lane number, computed anew: values made from it are not kept in registers
// over the loops
__device__ inline int lane_id() {
  int v;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(v));
  return v;
}

// asynchronous 4-byte copy of 64 lanes to 256 bytes of LDS
__device__ inline void dma4s(u32x4 rs, uint32_t voff, uint32_t soff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(m0), "v"(voff), "s"(rs), "s"(soff) : "memory");
}

// WIDE: out's rows start on 16 bytes
template <bool BF16, bool WIDE>
__global__ __launch_bounds__(256, 1) void mm_int_big_kernel(const IntMmParams p) {
  constexpr int BM = 256, BK = 128, STAGE = 2 * BM * BK, AHEAD = 1;
  constexpr int E = BF16 ? 2 : 4;                       // bytes per output
  constexpr int PITCH = 128 + 16;                       // a staged token: 128 bytes of outputs
  constexpr int NST = 16 * E;                           // stores of a tile (per thread)
  __shared__ __attribute__((aligned(16))) unsigned char lds[2 * STAGE];
  __shared__ __attribute__((aligned(16))) unsigned char stage_out[4 * 32 * PITCH];
  __shared__ __attribute__((aligned(16))) float scales[2][2 * BM];   // of w, then q, by tile parity
  __shared__ __attribute__((aligned(16))) uint32_t touched[BM];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w >> 1, wn = w & 1;

  IntTiles g;
  g.ntm1 = (p.N + 255) / 256;
  g.ntm = p.mats * g.ntm1;
  const int ntn = (int)((p.T + 255) / 256);
  g.ntiles = g.ntm * ntn;
  g.gsize = 4 * ntn;
  g.slots = gridDim.x >> 3;
  // tiles of an XCD (workgroup ids go round the XCDs) are consecutive; its workgroups take them in turn
  const int per_xcd = (g.ntiles + 7) / 8, first = (int)(blockIdx.x & 7) * per_xcd;
  g.last = min(first + per_xcd, g.ntiles);
  int tile = first + (int)(blockIdx.x >> 3);
  if (tile >= g.last) return;
  auto after = [&](int t) __attribute__((always_inline)) {
    return t + g.slots < g.last ? t + g.slots : g.ntiles;   // ntiles: no tile, its copies read zeros
  };
  const int nk = (p.K + BK - 1) / BK;

  // copy c of 16 of a step: rows 32 (c / 2) + 8 w + l / 8 of w (c even) or q (c
  // odd), chunk x of row r in slot x ^ swz(r)
  const int kc = 16 * ((l & 7) ^ swz<8>(8 * w + (l >> 3)));
  const uint32_t voff = (uint32_t)((8 * w + (l >> 3)) * p.K + kc), rows32 = 32u * (uint32_t)p.K;
  const uint32_t lds0 = lds_addr(lds) + (uint32_t)w * 1024u;
  IntPanels cp;                                           // the copies' tile, step and parity
  int cp_tile = tile;
  int cp_k = 0, cp_par = 0;
  cp.set(p, g, cp_tile);
  auto issue = [&](int buf, int c) __attribute__((always_inline)) {
    const uint32_t soff = __builtin_amdgcn_readfirstlane((uint32_t)(cp_k * BK));
    const uint32_t v = cp_k * BK + kc >= p.K ? kOutOfRange : voff + (uint32_t)(c >> 1) * rows32;
    dma16s(c & 1 ? cp.q : cp.w, v, soff, lds0 + (uint32_t)(buf * STAGE + (c & 1) * BM * BK + (c >> 1) * 4096));
  };
  // the scales of the copies' tile (issued with its first step)
  auto issue_scales = [&]() __attribute__((always_inline)) {
    const bool none = cp_tile >= g.ntiles;
    const int64_t sb = none ? 0 : (int64_t)(p.N - cp.n0) * 4, qb = none ? 0 : (p.T - (int64_t)cp.ti * 256) * 4;
    const uint32_t m0 = lds_addr(scales[cp_par]) + (uint32_t)w * 256u;
    dma4s(uniform_rsrc((cp.z ? p.w_scale[1] : p.w_scale[0]) + (none ? 0 : cp.n0), sb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)sb),
          (uint32_t)tid * 4, 0u, m0);
    dma4s(uniform_rsrc(p.q_scale + (none ? 0 : (int64_t)cp.ti * 256), qb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)qb),
          (uint32_t)tid * 4, 0u, m0 + 4 * BM);
  };
  auto next_copy = [&]() __attribute__((always_inline)) {
    if (++cp_k == nk) {
      cp_k = 0;
      cp_par ^= 1;
      cp_tile = after(cp_tile);
      cp.set(p, g, cp_tile);
    }
  };
  // touch: a 4-byte load to LDS (never read) of each line of this workgroup's
  // share of a step: 32 rows of w (waves 0, 1), which 8 neighbours have in
  // common, and 64 rows of q (waves 2, 3), which 4 have
  const uint32_t lds_t = lds_addr(touched) + (uint32_t)w * 256u;
  IntPanels tc;
  int tc_tile = tile;
  int tc_k = 0;
  uint32_t toff = 0;
  auto touch_tile = [&]() __attribute__((always_inline)) {
    tc.set(p, g, tc_tile);
    const int i = lane_id(), row = w < 2 ? 32 * (tc.ti % 8) + 16 * w + i : 64 * tc.ni + 32 * (w - 2) + i;
    toff = i < (w < 2 ? 16 : 32) ? (uint32_t)(row * p.K) : kOutOfRange;
  };
  auto next_touch = [&]() __attribute__((always_inline)) {
    if (++tc_k == nk) {
      tc_k = 0;
      tc_tile = after(tc_tile);
      touch_tile();
    }
  };
  auto touch = [&]() __attribute__((always_inline)) {
    dma4s(w < 2 ? tc.w : tc.q, toff,
          __builtin_amdgcn_readfirstlane((uint32_t)(tc_k * BK)), lds_t);
  };

  i32x16 acc[4][4];
  uint4 fa[2][4], fb[2][4];
  const int sl = swz<8>(l & 31), up = l >> 5;
  const int ra = (wm * 128 + (l & 31)) * BK, rb = (BM + wn * 128 + (l & 31)) * BK;
  // fragment f of 8 (4 of the channels, 4 of the tokens) of quarter h of a stage
  auto rd = [&](int buf, auto h, int f) __attribute__((always_inline)) {
    const unsigned char* sb = lds + buf * STAGE + (((2 * h + up) ^ sl) << 4);
    if (f < 4) fa[h & 1][f] = *reinterpret_cast<const uint4*>(sb + ra + f * 32 * BK);
    else fb[h & 1][f - 4] = *reinterpret_cast<const uint4*>(sb + rb + (f - 4) * 32 * BK);
  };
  // the 16 MFMAs of quarter h, behind(i) right behind the i-th
  auto mm = [&](auto quarter, auto behind) __attribute__((always_inline)) {
    constexpr int h = decltype(quarter)::value & 1;
    static_for<0, 16>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      mma_int(acc[i / 4][i % 4], fa[h][i / 4], fb[h][i % 4]);
      behind(ic);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  constexpr std::integral_constant<int, 0> Q0{};
  constexpr std::integral_constant<int, 1> Q1{};
  constexpr std::integral_constant<int, 2> Q2{};
  constexpr std::integral_constant<int, 3> Q3{};

  issue_scales();
#pragma unroll
  for (int c = 0; c < 16; ++c) issue(0, c);
  next_copy();
#pragma unroll
  for (int c = 0; c < 16; ++c) issue(1, c);
  next_copy();
  touch_tile();
#pragma unroll
  for (int s = 0; s < 2; ++s) next_touch();
#pragma unroll
  for (int s = 0; s < AHEAD; ++s) {
    touch();
    next_touch();
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(16 + AHEAD));       // the first step and its scales are in
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);

  int buf = 0, par = 0;
  bool stored = false;                                    // the previous tile's stores may be in flight
  while (true) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = i32x16{};
#pragma unroll
    for (int f = 0; f < 8; ++f) rd(buf, Q0, f);           // not kept over the epilogue
    for (int kt = 0; kt < nk; ++kt) {
      mm(Q0, [&](auto i) __attribute__((always_inline)) {
        if constexpr (i < 8) rd(buf, Q1, i);
      });
      mm(Q1, [&](auto i) __attribute__((always_inline)) {
        if constexpr (i < 8) rd(buf, Q2, i);
        if constexpr (i == 8) touch();
      });
      next_touch();
      mm(Q2, [&](auto i) __attribute__((always_inline)) {
        if constexpr (i < 8) rd(buf, Q3, i);
      });
      // step g + 1's copies are older than the touch of this step and, in a
      // tile's first step, than the stores of the tile before
      if (kt == 0 && stored) {
        constexpr int N1 = NST + 1 > 63 ? 63 : NST + 1;
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N1) : "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(1) lgkmcnt(0)" ::: "memory");
      }
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      if (cp_k == 0) issue_scales();
      mm(Q3, [&](auto i) __attribute__((always_inline)) {
        if constexpr (i < 8) rd(buf ^ 1, Q0, i);
        issue(buf, i);
      });
      next_copy();
      buf ^= 1;
    }

    // lane l holds token (l & 31) and channels 8 a + 4 (l / 32) + e of each 32 x
    // 32 tile: scaled, rounded and staged through LDS, 32 tokens x 128 bytes at a
    // time, so that out is written in whole lines
    const int le = lane_id();
    IntPanels here;
    here.set(p, g, tile);
    const int64_t t0 = (int64_t)here.ti * 256 + wn * 128;
    const int n0 = here.n0 + wm * 128;
    unsigned char* stg = stage_out + w * 32 * PITCH;
    const float* sw = scales[par] + wm * 128;
    const float* sq = scales[par] + BM + wn * 128;
    constexpr int CH = 128 / E / 32, G = 16 / CH;         // 32-channel tiles per 128 bytes; steps of the epilogue
    typedef std::conditional_t<BF16, uint2, float4> Four; // 4 outputs
    Four vals[CH * 4];
    // step s: tokens 32 (s CH / 4) .., channels 32 (s CH % 4) ..
    auto make = [&](auto sc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value, j = s * CH / 4, i0 = s * CH % 4;
      const float st = sq[j * 32 + (le & 31)];
#pragma unroll
      for (int i = i0; i < i0 + CH; ++i)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const float4 s4 = *reinterpret_cast<const float4*>(sw + i * 32 + 8 * a + 4 * (le >> 5));
          const float f[4] = {(float)acc[i][j][4 * a] * st * s4.x, (float)acc[i][j][4 * a + 1] * st * s4.y,
                              (float)acc[i][j][4 * a + 2] * st * s4.z, (float)acc[i][j][4 * a + 3] * st * s4.w};
          if constexpr (BF16) vals[(i - i0) * 4 + a] = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
          else vals[(i - i0) * 4 + a] = make_float4(f[0], f[1], f[2], f[3]);
        }
    };
    make(std::integral_constant<int, 0>{});
    static_for<0, G>([&](auto sc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value, j = s * CH / 4, i0 = s * CH % 4;
      const int64_t tj = t0 + j * 32;
      const int64_t rows = min<int64_t>(32, p.T - tj), ob = rows > 0 ? rows * p.N * E : 0;
      const __amdgpu_buffer_rsrc_t ro = buffer_rsrc(static_cast<unsigned char*>(here.z ? p.out[1] : p.out[0]) + (rows > 0 ? tj * p.N * E : 0), (uint32_t)ob);
      const int nb = n0 + i0 * 32;                        // the first of 128 / E channels
#pragma unroll
      for (int x = 0; x < CH * 4; ++x)
        *reinterpret_cast<Four*>(stg + (le & 31) * PITCH + (8 * x + 4 * (le >> 5)) * E) = vals[x];
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (WIDE) {
        u32x4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const u32x4*>(stg + (k * 8 + (le >> 3)) * PITCH + (le & 7) * 16);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (s + 1 < G) make(std::integral_constant<int, s + 1 < G ? s + 1 : 0>{});   // while the reads run
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = k * 8 + (le >> 3), n = nb + (le & 7) * (16 / E);
          const uint32_t off = n < p.N ? (uint32_t)(row * p.N + n) * E : 0xfffffff0u;
          __builtin_amdgcn_raw_buffer_store_b128(v[k], ro, (int)off, 0, 2);   // non-temporal: the panels stay in L2
        }
      } else {
        if constexpr (!BF16) {
          for (int k = 0; k < 16; ++k) {
            const int row = k * 2 + (le >> 5), n = nb + (le & 31);
            const uint32_t v = *reinterpret_cast<const uint32_t*>(stg + row * PITCH + (le & 31) * 4);
            const uint32_t off = n < p.N ? (uint32_t)(row * p.N + n) * 4u : 0xfffffff0u;
            __builtin_amdgcn_raw_buffer_store_b32(v, ro, (int)off, 0, 0);
          }
        } else {
          // rows that start on any element: pairs that lie on 4 bytes, and the
          // elements left at both ends
          const int m = min(64, p.N - nb);
          for (int k = 0; k < 16; ++k) {
            const int row = k * 2 + (le >> 5), odd = (int)((tj + row) & p.N & 1), c = 2 * (le & 31) + odd;
            const uint16_t* s = reinterpret_cast<const uint16_t*>(stg + row * PITCH) + c;
            const uint32_t v = (uint32_t)s[0] | ((uint32_t)s[1] << 16);
            const uint32_t off = c + 1 < m ? (uint32_t)(row * p.N + nb + c) * 2u : 0xfffffff0u;
            __builtin_amdgcn_raw_buffer_store_b32(v, ro, (int)off, 0, 0);
          }
          const int row = le & 31, odd = (int)((tj + row) & p.N & 1), c = le < 32 ? 0 : m - 1;
          if (m > 0) {
            const uint16_t v = reinterpret_cast<const uint16_t*>(stg + row * PITCH)[c];
            const bool on = le < 32 ? odd : (m - odd) & 1;
            __builtin_amdgcn_raw_buffer_store_b16(v, ro, on ? (int)((uint32_t)(row * p.N + nb + c) * 2u) : (int)0xfffffff0u, 0, 0);
          }
        }
        if constexpr (s + 1 < G) make(std::integral_constant<int, s + 1 < G ? s + 1 : 0>{});
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (WIDE) stored = true;
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // a varying number of stores
    tile = after(tile);
    if (tile >= g.ntiles) break;
    par ^= 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <int BM, int BN, int WGM, int WGN, int KG, int NST>
hipError_t launch_t(const IntMmParams& p, hipStream_t st) {
  const int64_t ntiles = (int64_t)((p.N + BM - 1) / BM) * ((p.T + BN - 1) / BN);
  const dim3 grid((unsigned)(8 * ((ntiles + 7) / 8)), p.mats);
  hipLaunchKernelGGL((mm_int_kernel<BM, BN, WGM, WGN, KG, NST>), grid, dim3(64 * WGM * WGN * KG), 0, st, p);
  return hipGetLastError();
}

// Up to 16 tokens: bound by the weights' bytes (one token) or by latency.  A
// workgroup holds 16 channels against all tokens, its W waves each a part of k,
// straight from memory into 16 x 16 x 64 MFMA operands: nothing is shared, so
// LDS only joins the waves' sums (int32: exact in any order).  Rows past N or T
// are read from the last one and not written.
template <int W>
__global__ __launch_bounds__(64 * W) void mm_int_few_kernel(const IntMmParams p) {
  constexpr int UN = 8;                                   // 64-byte steps of k in flight
  __shared__ int part[W][4][64];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int n0 = blockIdx.x * 16, kl = 16 * (l >> 4);
  const int8_t* pa = (blockIdx.y ? p.w[1] : p.w[0]) + (int64_t)min(n0 + (l & 15), p.N - 1) * p.K;
  const int8_t* pb = p.q + (int64_t)min(l & 15, (int)p.T - 1) * p.K;
  i32x4 acc = {};
  const int steps = (p.K + 63) / 64, per = (steps + W - 1) / W;
  const int s1 = min(steps, (w + 1) * per);
  for (int s = w * per; s < s1; s += UN) {
    uint4 a[UN], b[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int k = (s + u) * 64 + kl;
      const bool on = s + u < s1 && k < p.K;              // zeros of w where this wave's part or k ends
      a[u] = make_uint4(0, 0, 0, 0);
      if (on) a[u] = *reinterpret_cast<const uint4*>(pa + k);
      b[u] = *reinterpret_cast<const uint4*>(pb + (on ? k : 0));
    }
#pragma unroll
    for (int u = 0; u < UN; ++u)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a[u]), __builtin_bit_cast(i32x4, b[u]), acc, 0, 0, 0);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) part[w][e][l] = acc[e];
  __syncthreads();
  if (w > 0) return;
  // lane l holds token l & 15 and channels 4 (l / 16) + e
  int v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = part[0][e][l];
#pragma unroll
    for (int x = 1; x < W; ++x) v[e] += part[x][e][l];
  }
  const int t = l & 15, n = n0 + 4 * (l >> 4);
  if (t < p.T && n < p.N) put4(p, blockIdx.y, t, n, v, p.q_scale[t]);
}

// 8 waves a workgroup where there is at most one workgroup a CU and k is long,
// else 4.  One token, weights read from HBM, us with 4 and 8 (and 16) waves:
// 4096 x 4096 6.4, 6.1 (6.8), 4096 x 14336 16.8, 14.2 (14.4); 4096 x 2048 4.1,
// 4.6 (5.1); 5120 x 4096 8.3, 8.3 (10.0), 6144 x 14336 21.7, 23.3 (23.9), 28672 x 4096
// 22.2, 22.7 (30.5).
hipError_t launch_few(const IntMmParams& p, hipStream_t st) {
  const dim3 grid((p.N + 15) / 16, p.mats);
  if ((int64_t)grid.x * p.mats <= 256 && p.K > 2048) hipLaunchKernelGGL(mm_int_few_kernel<8>, grid, dim3(512), 0, st, p);
  else hipLaunchKernelGGL(mm_int_few_kernel<4>, grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_int(const IntMmParams& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  // Variants, by the tiles they make of the outputs (T x N, or twice that) on 256 CUs; times in us of both
  // sides of each border.
  auto tiles = [&](int m, int n) { return p.mats * (int64_t)((p.N + m - 1) / m) * ((p.T + n - 1) / n); };
  // No LDS for up to 4 tokens, whatever the weights: 1 token, weights read from
  // HBM, against the best tiles: 4096 x 4096 6.1 (7.5 with 32 x 32), 14336 x 4096
  // 13.9 (15.1 with 64 x 64), 40960 x 4096 32 (39 with 64 x 64, 58 with 256 x 256),
  // 65536 x 1024 15.7 (22.6, 23.1); behind where 32 x 32 or 64 x 64 make one round and k is long:
  // 6144 x 14336 21.7 (18.6), 14336 x 14336 42 (37).  At 4 and 5 tokens 4096 x 4096
  // 6.3 (7.6) and 6.4 (7.7), 14336 x 4096 15.3 (15.2) and 16.6 (15.0).
  if (p.T <= 4) return launch_few(p, st);
  // 256 x 256 from 160 tiles on.  T x N x K 4096 x 2531 x 1008 (160 tiles): 27
  // against 34 with 128 x 128; 2048 x 4096 x 1024 (128 tiles): 20 against 17.
  // Two steps a tile at least: its scales are in before the tile before it ends.
  if (tiles(256, 256) >= 160 && p.K > 128) {
    auto go = [&](auto bf16, auto wide) {
      hipLaunchKernelGGL((mm_int_big_kernel<decltype(bf16)::value, decltype(wide)::value>), dim3(256), dim3(256), 0, st, p);
    };
    if (p.out_bf16 && p.N % 8 == 0) go(std::true_type{}, std::true_type{});
    else if (p.out_bf16) go(std::true_type{}, std::false_type{});
    else if (p.N % 4 == 0) go(std::false_type{}, std::true_type{});
    else go(std::false_type{}, std::false_type{});
    return hipGetLastError();
  }
  // No LDS for up to 16 with short k either: 16 tokens, 4096 x 1024 4.1 against 4.8
  // with 32 x 32 tiles (14336 x 1024 8.6 against 6.4 with 64 x 64); 4096 x 2048 4.9 against
  // 6.0, 14336 x 2048 11.4 against 9.1.
  if (p.T <= 16 && p.K <= 1024) return launch_few(p, st);
  // 32 x 32 with k in four while they are one round: 4096 x 14336 weights, 64
  // tokens (256 tiles) 15 against 23 with 64 x 64, 128 tokens 27 against 24.
  const int64_t t64 = tiles(64, 64);
  if (tiles(32, 32) <= 256) return launch_t<32, 32, 1, 1, 4, 4>(p, st);
  // 64 x 64 with k in two up to two rounds, four stages for one round of long k: T x N
  // x K 128 x 4096 x 14336 37 against 50 with two stages; 300 x 2531 (200 tiles) x 2048
  // 8.7 against 10.5, x 1024 6.1 against 6.2, x 784 6.8 against 6.5, x 272 5.5 against
  // 5.2; 512 x 4096 x 14336 (two rounds) 56 against 52.  512 x 4096 x 1024 6.9 against
  // 8.5 with 128 x 128, 1024 tokens (four rounds) 13.2 against 10.8.
  if (t64 <= 256 && p.K >= 1024) return launch_t<64, 64, 2, 2, 2, 4>(p, st);
  if (t64 <= 512) return launch_t<64, 64, 2, 2, 2, 2>(p, st);
  // 128 x 128, k in two for one round: 4096 x 14336, 1024 tokens (256 tiles) 69
  // to 83 against 79 to 95, 1500 tokens (384 tiles) 138 against 109.
  if (tiles(128, 128) <= 256) return launch_t<128, 128, 2, 2, 2, 2>(p, st);
  return launch_t<128, 128, 2, 2, 1, 2>(p, st);
}

}  // namespace hna
