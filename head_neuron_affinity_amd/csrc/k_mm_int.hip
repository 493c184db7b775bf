// 8-bit integer product on the matrix cores:
//   out[t, n] = (sum_k q[t, k] w[n, k]) q_scale[t] w_scale[n]
// q [T, K] and w [N, K] row-major with k contiguous, sums in int32 (exact for
// K < 2^17), the scales applied in fp32, one rounding to the output type.
// The channels are the MFMA rows and the tokens its columns, so a lane ends up
// with 4 consecutive channels of one token: out's contiguous direction.
// Tiles of 128 x 128 on 4 waves, 128 bytes of k a step through LDS.
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
__device__ inline void put4(const IntMmParams& p, int64_t t, int n, const int (&v)[4], float st) {
  const int64_t o = t * p.N + n;
  if (n + 4 <= p.N && p.N % 4 == 0) {
    const float4 sw = *reinterpret_cast<const float4*>(p.w_scale + n);
    const float f[4] = {(float)v[0] * st * sw.x, (float)v[1] * st * sw.y, (float)v[2] * st * sw.z, (float)v[3] * st * sw.w};
    if (p.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(f[0], f[1], f[2], f[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p.N) break;
    const float f = (float)v[e] * st * p.w_scale[n + e];
    if (p.out_bf16) static_cast<uint16_t*>(p.out)[o + e] = (uint16_t)pack_bf16x2(f, 0.f);
    else static_cast<float*>(p.out)[o + e] = f;
  }
}

template <int BM, int BN, int WGM, int WGN, int NST>
__global__ __launch_bounds__(64 * WGM * WGN) void mm_int_kernel(const IntMmParams p) {
  constexpr int NW = WGM * WGN;
  constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  constexpr int ROWS = BM + BN, BK = 128, CPR = BK / 16, RPI = 64 / CPR;
  constexpr int STAGE = ROWS * BK;
  constexpr int NCP = ROWS / (RPI * NW), NCX = BM / (RPI * NW);
  static_assert(BM % (RPI * NW) == 0 && BN % (RPI * NW) == 0, "copy rounds cover whole rows");
  static_assert((NST - 2) * NCP <= 63, "copies in flight must fit the wait counter");
  __shared__ __attribute__((aligned(16))) unsigned char lds[NST * STAGE];

  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WGN, wn = w % WGN;

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
  const u32x4 rx = uniform_rsrc(p.w + (int64_t)n0 * p.K, xb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)xb);
  const u32x4 ry = uniform_rsrc(p.q + t0 * p.K, yb > kMaxResourceBytes ? kMaxResourceBytes : (uint32_t)yb);

  i32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x16{};
  const int nk = (p.K + BK - 1) / BK;

  // copy i of wave w fills rows RPI (NW i + w) .. + RPI - 1 of the stage (w
  // rows first); rows past the end and bytes past K read zeros
  uint32_t voff[NCP];
  int kc[NCP];
#pragma unroll
  for (int i = 0; i < NCP; ++i) {
    const int r = RPI * (NW * i + w) + l / CPR;
    kc[i] = 16 * ((l % CPR) ^ swz<CPR>(r));
    voff[i] = (uint32_t)((int64_t)(i < NCX ? r : r - BM) * p.K + kc[i]);
  }
  const uint32_t lds0 = lds_addr(lds) + (uint32_t)w * 1024u;
  auto issue = [&](int k0, int buf) __attribute__((always_inline)) {
    const uint32_t base = lds0 + (uint32_t)(buf * STAGE);
    const uint32_t soff = __builtin_amdgcn_readfirstlane((uint32_t)k0);
#pragma unroll
    for (int i = 0; i < NCP; ++i)
      dma16s(i < NCX ? rx : ry, k0 + kc[i] >= p.K ? kOutOfRange : voff[i], soff, base + (uint32_t)(i * NW * 1024));
  };

#pragma unroll
  for (int st = 0; st < NST - 1; ++st)
    if (st < nk) issue(st * BK, st);
  for (int kt = 0; kt < nk; ++kt) {
    // step kt has landed once at most the copies of the steps after it are in
    // flight; the barrier shows it to every wave and ends their reads of step kt - 1
    const int ahead = min(NST - 2, nk - 1 - kt);
    if (NST >= 4 && ahead >= 2) __builtin_amdgcn_s_waitcnt(vm_wait(2 * NCP));
    else if (NST >= 3 && ahead >= 1) __builtin_amdgcn_s_waitcnt(vm_wait(NCP));
    else __builtin_amdgcn_s_waitcnt(vm_wait(0));
    __syncthreads();
    if (kt + NST - 1 < nk) issue((kt + NST - 1) * BK, (kt + NST - 1) % NST);
    const unsigned char* sb = lds + (kt % NST) * STAGE;
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
  }

  // lane l holds token (l & 31) and channels 8 (v / 4) + 4 (l / 32) + v % 4 of each tile
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t tk = t0 + wn * WN + j * 32 + (l & 31);
    if (tk >= p.T) continue;
    const float st = p.q_scale[tk];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int n = n0 + wm * WM + i * 32 + 8 * a + 4 * (l >> 5);
        if (n >= p.N) continue;
        const int v[4] = {acc[i][j][4 * a], acc[i][j][4 * a + 1], acc[i][j][4 * a + 2], acc[i][j][4 * a + 3]};
        put4(p, tk, n, v, st);
      }
  }
}

template <int BM, int BN, int WGM, int WGN, int NST>
hipError_t launch_t(const IntMmParams& p, hipStream_t st) {
  const int64_t ntiles = (int64_t)((p.N + BM - 1) / BM) * ((p.T + BN - 1) / BN);
  const dim3 grid((unsigned)(8 * ((ntiles + 7) / 8)));
  hipLaunchKernelGGL((mm_int_kernel<BM, BN, WGM, WGN, NST>), grid, dim3(64 * WGM * WGN), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_int(const IntMmParams& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  return launch_t<128, 128, 2, 2, 2>(p, st);
}

}  // namespace hna
