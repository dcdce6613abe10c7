// Gated delta rule, backward, for gfx950.
#include "gdr_tile.h"

namespace ssmb {
namespace {

// ---------------------------------------------------------------------------
// From chunk to chunk, the last one first: dS, and E = T^T dU, dv = beta E
// ---------------------------------------------------------------------------

// As in the forward two wavefronts carry dS, 16 columns each, and two others
// make what does not depend on it, A^T dY and Q^T (scale e^G dY), copy the next
// chunk, and store E and dv.
template <int KD>
__global__ void __launch_bounds__(256) gdr_bwd_kernel(const GdrParams p) {
  constexpr int NT = 64 * kPairs, NC = 16 * kPairs, NS = KD / 32, NB = KD / 16;
  constexpr unsigned kRows = 64 * KD * 2, kValues = 64 * NC * 2, kTri = 2 * kGdrTriBytes, kOps = kTri + kGdrGateBytes;
  constexpr unsigned kAtQ = kRows, kAtD = 2 * kRows, kAtW = kAtD + kValues, kBuffer = kAtW + kOps;
  constexpr unsigned kFour = 4 * 1024, kState = NB * 1024;  // float32 D results of the tokens, and of the state
  __shared__ __align__(16) u4 lds[(2 * kBuffer + kPairs * (kFour + kState)) / 16];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave % kPairs;
  const HeadTile which = head_tile(blockIdx.x, static_cast<unsigned>(p.batch * p.nheads), static_cast<unsigned>(p.vdim) / NC);
  const int64_t vt = which.tile, bh = which.head, b = bh / p.nheads, h = bh % p.nheads;
  const int len = gdr_length(p.lengths, b, p.seqlen), n = (len + 63) / 64;
  const int col0 = static_cast<int>(vt) * NC + 16 * w;
  const unsigned base = lds_at(lds), four = base + 2 * kBuffer + w * kFour + lane * 16;
  const unsigned grown = base + 2 * kBuffer + kPairs * kFour + w * kState + lane * 16;
  const Lanes16 at = lanes16_of<KD>(lane);
  typedef __attribute__((address_space(3))) f4v lds_f4v;

  if (wave < kPairs) {
    f4v s[NB];  // dS, laid out as the state
    const int64_t state = (bh * p.vdim + col0 + m) * KD + 8 * g;
#pragma unroll
    for (int j = 0; j < NB; ++j)
      s[j] = p.dh_last != nullptr ? *reinterpret_cast<const f4v *>(p.dh_last + state + 32 * (j / 2) + 4 * (j % 2)) : f4v{};
    for (int c = n - 1; c >= 0; --c) {
      float *to = p.ws_ds + ((bh * p.chunks + c) * p.vdim + col0 + m) * KD + 8 * g;
#pragma unroll
      for (int j = 0; j < NB; ++j) *reinterpret_cast<f4v *>(to + 32 * (j / 2) + 4 * (j % 2)) = s[j];
      Parts sp[NS];
#pragma unroll
      for (int a = 0; a < NS; ++a) sp[a] = parts(s[2 * a], s[2 * a + 1]);
      meet();
      const unsigned tile = base + (c & 1) * kBuffer, at_t = tile + kAtW, gates = at_t + kTri + 16 * g;
      bf8 ka[NS][4], kt[2][NB];
      Parts tf[kGdrFrags];
      f4v out[4], fac[4];
#pragma unroll
      for (int a = 0; a < NS; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) ka[a][i] = row16<KD>(tile, i, a, at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        out[i] = lds_f4(gates + 512 + 64 * i);
        fac[i] = lds_f4(gates + 256 + 64 * i) * -lds_f4(gates + 768 + 64 * i);
      }
#pragma unroll
      for (int f = 0; f < kGdrFrags; ++f) tf[f] = {frag16(at_t, f, lane), frag16(at_t, kGdrFrags + f, lane)};
      const float whole = lds_f4(at_t + kTri + 256 + 240)[3];
      __builtin_amdgcn_sched_barrier(0);
      // K dS, and dU = e^(GC - G) of that + A^T dY
      f4v x[4] = {};
#pragma unroll
      for (int a = 0; a < NS; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul_exact(ka[a][i], sp[a], x[i]);
      meet();
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = x[i] * out[i] + *(const lds_f4v *)(four + i * 1024);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NB; ++j) kt[k][j] = col16<KD>(tile, j, k, at);
      // E = T^T dU
      f4v e[4] = {};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Parts xp = parts(x[2 * k], x[2 * k + 1]);
#pragma unroll
        for (int j = 0; j <= 2 * k + 1; ++j) e[j] = mul_parts(tf[tri_t(j, k)], xp, e[j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) *(lds_f4v *)(four + i * 1024) = e[i];
      const Parts ep[2] = {parts(e[0] * fac[0], e[1] * fac[1]), parts(e[2] * fac[2], e[3] * fac[3])};
      meet();
      // dS = e^GC dS + sum over tokens of q (scale e^G dy) - k (e^G beta E)
#pragma unroll
      for (int j = 0; j < NB; ++j) s[j] = s[j] * whole + *(const lds_f4v *)(grown + j * 1024);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NB; ++j) s[j] = mul_exact(kt[k][j], ep[k], s[j]);
    }
    if (p.dh0 != nullptr) {
#pragma unroll
      for (int j = 0; j < NB; ++j) *reinterpret_cast<f4v *>(p.dh0 + state + 32 * (j / 2) + 4 * (j % 2)) = s[j];
    }
    return;
  }

  const int id = tid - NT;
  const int64_t hk = h / (p.nheads / p.nqk), yt = p.nheads * p.vdim;
  const uint16_t *kp = p.k + b * p.k_batch + hk * KD, *qp = p.q + b * p.q_batch + hk * KD;
  const uint16_t *dp = p.dy + (b * p.seqlen * p.nheads + h) * p.vdim + vt * NC;
  const char *ws = p.ws + bh * p.chunks * static_cast<int64_t>(kGdrBwdChunkBytes) + kGdrTriBytes;  // T^T, A^T, gates
  uint16_t *vp = p.dv + (b * p.seqlen * p.nheads + h) * p.vdim + col0;
  TileCopy<KD, NT> k_copy, q_copy;
  TileCopy<NC, NT> d_copy;
  k_copy.init(p.k_token, id);
  q_copy.init(p.q_token, id);
  d_copy.init(yt, id);
  RowStore v_store;
  v_store.init(yt, lane);
  auto fetch_rows = [&](int c) {
    u4 *to = lds + (c & 1) * (kBuffer / 16);
    const int last = len - 1 - 64 * c;
    k_copy.start(to, kp + 64 * c * p.k_token, last, id);
    q_copy.start(to + kAtQ / 16, qp + 64 * c * p.q_token, last, id);
    d_copy.start(to + kAtD / 16, dp + 64 * c * yt, last, id);
  };
  auto fetch_ws = [&](int c) {
    copy_share<kOps / 1024, kPairs>(base + (c & 1) * kBuffer + kAtW, ws + c * static_cast<int64_t>(kGdrBwdChunkBytes), w, lane * 16);
  };
  f4v e[4];
  auto store = [&](int c) {
    float *to = p.ws_e + (bh * p.chunks + c) * 64 * p.vdim + (vt * kPairs + w) * 1024 + lane * 4;
    const unsigned beta = base + (c & 1) * kBuffer + kAtW + kTri + 768 + 16 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<f4v *>(to + i * 256) = e[i];
      e[i] *= lds_f4(beta + 64 * i);
    }
    if (64 * c + 64 > len) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (64 * c + 16 * i + 4 * g + r >= len) e[i][r] = 0.0f;
    }
    const int64_t rest = p.seqlen - 64 * static_cast<int64_t>(c);
    v_store.put(vp + 64 * c * yt, rest < 64 ? static_cast<int>(rest) : 64, e);
  };
  if (n > 0) {
    fetch_rows(n - 1);
    fetch_ws(n - 1);
  }
  for (int c = n - 1; c >= 0; --c) {
    arrive();
    const unsigned tile = base + (c & 1) * kBuffer, at_a = tile + kAtW + kGdrTriBytes, gates = at_a + kGdrTriBytes + 16 * g;
    Parts af[kGdrFrags];
    sh4 dy[4];
    bf8 qt[2][NB];
#pragma unroll
    for (int i = 0; i < 4; ++i) dy[i] = rows4<NC>(tile + kAtD, i, w, lane);
#pragma unroll
    for (int f = 0; f < kGdrFrags; ++f) af[f] = {frag16(at_a, f, lane), frag16(at_a, kGdrFrags + f, lane)};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < NB; ++j) qt[k][j] = col16<KD>(tile + kAtQ, j, k, at);
    __builtin_amdgcn_sched_barrier(0);
    f4v x[4] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bf8 d = __builtin_bit_cast(bf8, __builtin_shufflevector(dy[2 * k], dy[2 * k + 1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int j = 0; j <= 2 * k + 1; ++j) x[j] = mfma16(af[tri_t(j, k)].hi, d, mfma16(af[tri_t(j, k)].lo, d, x[j]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) *(lds_f4v *)(four + i * 1024) = x[i];
    meet();
    if (c > 0) fetch_rows(c - 1);
    f4v z[NB] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      f4v y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f4v qs = lds_f4(gates + 64 * (2 * k + i));
#pragma unroll
        for (int r = 0; r < 4; ++r) y[i][r] = up(dy[2 * k + i][r]) * qs[r];
      }
      const Parts yp = parts(y[0], y[1]);
#pragma unroll
      for (int j = 0; j < NB; ++j) z[j] = mul_exact(qt[k][j], yp, z[j]);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) *(lds_f4v *)(grown + j * 1024) = z[j];
    meet();
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = *(const lds_f4v *)(four + i * 1024);
    if (c > 0) fetch_ws(c - 1);
    store(c);
  }
  for (int64_t row = 64 * static_cast<int64_t>(n) + g; row < p.seqlen; row += 4) st(vp, row * yt + m, 0.0f);
}

// ---------------------------------------------------------------------------
// Within a chunk: dq, dk, dg, dbeta
// ---------------------------------------------------------------------------

// Transposed operands of a tile of 64-column rows [value][token], in two
// parts: lane m stands for token 16 i + m, k for values 32 s + 8g ..
struct Pair {
  unsigned hi, lo;  // where the tiles are
};
__device__ __forceinline__ bf8 tokens16(unsigned tile, int i, int s, unsigned col) {
  typedef __attribute__((address_space(3))) sh4 lds4;
  const unsigned to = ((tile + col) ^ (32 * i)) + s * 32 * 128;
  const sh4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(to));
  const sh4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)((to ^ 16) + 4 * 128));
  return __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ Parts tokens16(const Pair &t, int i, int s, unsigned col) {
  return {tokens16(t.hi, i, s, col), tokens16(t.lo, i, s, col)};
}

// Operand of the elements 16 ct + m of a row-major tile, k its rows 32 s .. in D's order.
template <int D>
__device__ __forceinline__ bf8 elems16(unsigned tile, int ct, int s, int lane) {
  return __builtin_bit_cast(bf8, __builtin_shufflevector(rows4<D>(tile, 2 * s, ct, lane), rows4<D>(tile, 2 * s + 1, ct, lane), 0,
                                                         1, 2, 3, 4, 5, 6, 7));
}

// The sum over the 16 lanes of a row.
__device__ __forceinline__ float sum16(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true));
  return v;
}

__device__ __forceinline__ void store_gate(void *p, int64_t i, float v, float) { st(static_cast<float *>(p), i, v); }
__device__ __forceinline__ void store_gate(void *p, int64_t i, float v, uint16_t) { st(static_cast<uint16_t *>(p), i, v); }

// A workgroup per chunk and query head, over the value heads that share it; a
// wavefront per 16 key elements.
template <int KD, int VD, typename G>
__global__ void __launch_bounds__(4 * KD) gdr_grad_kernel(const GdrParams p) {
  constexpr int NW = KD / 16, NT = 64 * NW, NS = KD / 32, NV = VD / 32;
  constexpr unsigned kRows = 64 * KD * 2, kAtQ = kRows, kAtD = 2 * kRows, kAtU = kAtD + 64 * VD * 2, kPart = VD * 128;
  constexpr unsigned kFour = 4 * (kPart > kGdrTriBytes ? kPart : kGdrTriBytes), kAtS = kAtU + kFour, kSlice = 32 * KD * 2;
  __shared__ __align__(16) u4 lds[(kAtS + 4 * kSlice) / 16];
  __shared__ float red[2][NW][64], whole[NW];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c = blockIdx.x % p.chunks, bk = blockIdx.x / p.chunks, b = bk / p.nqk, hk = bk % p.nqk;
  const int64_t share = p.nheads / p.nqk;
  const int t0 = static_cast<int>(c) * 64, len = gdr_length(p.lengths, b, p.seqlen) - t0;
  const int rows = p.seqlen - t0 < 64 ? static_cast<int>(p.seqlen - t0) : 64;
  f4v tq[4] = {}, tk[4] = {};
  if (len > 0) {
    const unsigned base = lds_at(lds);
    load_tile<KD, NT>(lds, p.k + b * p.k_batch + hk * KD, p.k_token, t0, t0 + len - 1, threadIdx.x);
    load_tile<KD, NT>(lds + kAtQ / 16, p.q + b * p.q_batch + hk * KD, p.q_token, t0, t0 + len - 1, threadIdx.x);
#pragma unroll 1
    for (int64_t h = hk * share; h < (hk + 1) * share; ++h) {
    // (Made anew for each head: the compiler would keep all that follows from
    // it, hundreds of addresses and masks, from one head to the next.)
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, m = lane & 15, g = lane >> 4;
    const Lanes16 atk = lanes16_of<KD>(lane), atv = lanes16_of<VD>(lane);
    // Where this lane's pieces of transposed reads lie: row 8g + m / 4, elements 4 (m % 4) ..
    const unsigned col = static_cast<unsigned>(slot<64>(8 * g + (m >> 2), (m & 3) >> 1)) * 16 + (m & 1) * 8;
    const unsigned col_s = (static_cast<unsigned>(slot<KD>(8 * g + (m >> 2), (m & 3) >> 1)) * 16 + (m & 1) * 8) ^ (32 * w);
    const Pair U = {base + kAtU, base + kAtU + kPart}, D = {base + kAtU + 2 * kPart, base + kAtU + 3 * kPart};
      const int64_t bh = b * p.nheads + h, id = bh * p.chunks + c, yt = p.nheads * VD;
      const char *ws = p.ws + id * static_cast<int64_t>(kGdrBwdChunkBytes);
      const float *gates = reinterpret_cast<const float *>(ws + 3 * kGdrTriBytes);
      const double *sums = reinterpret_cast<const double *>(gates + 256);
      const float *s0 = p.states + id * VD * KD, *ds0 = p.ws_ds + id * VD * KD;
      load_tile<VD, NT>(lds + kAtD / 16, p.dy + (b * p.seqlen * p.nheads + h) * VD, yt, t0, t0 + len - 1, tid);
      // Of 32 values at a time, this thread's 8 elements of the state and of dS.
      f4v sv[2], dv[2];
      auto fetch_slice = [&](int s) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          sv[k] = *reinterpret_cast<const f4v *>(s0 + s * 32 * KD + (k * NT + tid) * 4);
          dv[k] = *reinterpret_cast<const f4v *>(ds0 + s * 32 * KD + (k * NT + tid) * 4);
        }
      };
      // U = T beta (V - e^G K S0), a wavefront per 16 values; U and D = beta E go to LDS in parts.
      float db[4][4] = {};
#pragma unroll 1
      for (int ct = w; ct < VD / 16; ct += NW) {
        f4v sf[NS][2], e[4], beta[4], into[4];
        float vf[4][4];
        Parts tf[kGdrFrags];
        const float *from = s0 + (16 * ct + m) * KD + 8 * g;
#pragma unroll
        for (int a = 0; a < NS; ++a)
#pragma unroll
          for (int k = 0; k < 2; ++k) sf[a][k] = *reinterpret_cast<const f4v *>(from + 32 * a + 4 * k);
        const uint16_t *vp = p.v + b * p.v_batch + t0 * p.v_token + h * VD + 16 * ct + m;
        const u4 *tp = reinterpret_cast<const u4 *>(ws) + lane;
        const float *ep = p.ws_e + id * 64 * VD + ct * 1024 + lane * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          into[i] = *reinterpret_cast<const f4v *>(gates + 64 + 16 * i + 4 * g);
          beta[i] = *reinterpret_cast<const f4v *>(gates + 192 + 16 * i + 4 * g);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * i + 4 * g + r;
            vf[i][r] = ld(vp, (row < len ? row : len - 1) * p.v_token);
          }
        }
#pragma unroll
        for (int f = 0; f < kGdrFrags; ++f)
          tf[f] = {__builtin_bit_cast(bf8, tp[f * 64]), __builtin_bit_cast(bf8, tp[(kGdrFrags + f) * 64])};
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = *reinterpret_cast<const f4v *>(ep + i * 256);
        if (ct == w) arrive();  // keys, queries and dy are in LDS
        f4v x[4] = {};
#pragma unroll
        for (int a = 0; a < NS; ++a) {
          const Parts sp = parts(sf[a][0], sf[a][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = mul_exact(row16<KD>(base, i, a, atk), sp, x[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) x[i][r] = beta[i][r] * fmaf(-into[i][r], x[i][r], vf[i][r]);
        f4v u[4] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const Parts xp = parts(x[2 * k], x[2 * k + 1]);
#pragma unroll
          for (int i = 2 * k; i < 4; ++i) u[i] = mul_parts(tf[tri(i, k)], xp, u[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int r = 0; r < 4; ++r) db[i][r] = fmaf(e[i][r], u[i][r] / beta[i][r], db[i][r]);
          e[i] *= beta[i];
        }
        typedef __attribute__((address_space(3))) u2 lds8;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const Parts up = parts(u[2 * k], u[2 * k + 1]), dp = parts(e[2 * k], e[2 * k + 1]);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const unsigned to = static_cast<unsigned>(slot<64>(16 * ct + m, 2 * (2 * k + y) + (g >> 1))) * 16 + (g & 1) * 8;
            *(lds8 *)(U.hi + to) = half_of(up.hi, y);
            *(lds8 *)(U.lo + to) = half_of(up.lo, y);
            *(lds8 *)(D.hi + to) = half_of(dp.hi, y);
            *(lds8 *)(D.lo + to) = half_of(dp.lo, y);
          }
        }
      }
      if (w >= VD / 16) arrive();
      fetch_slice(0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v = sum16(db[i][r]);
          if (m == 0) red[0][w][16 * i + 4 * g + r] = v;
        }
      meet();
      // P = scale (dY U^T) M and H = -(D U^T) M within the chunk, and their transposes, as fragments.
      u4 frag[8 / NW][2][4];  // [P or H of this wavefront][as it is or transposed][parts of 2 steps]
      auto products = [&](auto wave, auto kind, u4 (&f)[2][4]) {
        constexpr int W = wave;
        constexpr bool HH = kind;
        f4v lower[W + 1] = {}, upper[4 - W] = {};
#pragma unroll 1
        for (int s = 0; s < NV; ++s) {
          const Parts uw = tokens16(U, W, s, col);
          const Parts dw = HH ? tokens16(D, W, s, col) : Parts{row16<VD>(base + kAtD, W, s, atv), bf8{}};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j <= W) {  // rows j, columns i = 16 W + m
              const Parts uj = j == W ? uw : tokens16(U, j, s, col);
              lower[j <= W ? j : 0] = HH ? mul_parts(uj, dw, lower[j <= W ? j : 0])
                                         : mfma16(uj.hi, dw.hi, mfma16(uj.lo, dw.hi, lower[j <= W ? j : 0]));
            }
            if (j >= W) {  // rows i, columns j = 16 W + m
              const Parts di = j == W ? dw : HH ? tokens16(D, j, s, col) : Parts{row16<VD>(base + kAtD, j, s, atv), bf8{}};
              upper[j >= W ? j - W : 0] = HH ? mul_parts(di, uw, upper[j >= W ? j - W : 0])
                                             : mul_exact(di.hi, uw, upper[j >= W ? j - W : 0]);
            }
          }
        }
        const int own = 16 * W + m;
        const double so = sums[own];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int other = 16 * j + 4 * g + r;
            const double st = sums[other];
            if (j <= W) {  // i = own, j = other
              const bool in = HH ? other < own : other <= own && own < len;
              const float f = (HH ? -1.0f : p.scale) * __builtin_amdgcn_exp2f(static_cast<float>(so - st));
              lower[j <= W ? j : 0][r] = in ? lower[j <= W ? j : 0][r] * f : 0.0f;
            }
            if (j >= W) {
              const bool in = HH ? own < other : own <= other && other < len;
              const float f = (HH ? -1.0f : p.scale) * __builtin_amdgcn_exp2f(static_cast<float>(st - so));
              upper[j >= W ? j - W : 0][r] = in ? upper[j >= W ? j - W : 0][r] * f : 0.0f;
            }
          }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const f4v zero = {};
          if (2 * s <= W) {
            const Parts x = parts(lower[2 * s <= W ? 2 * s : 0], 2 * s + 1 <= W ? lower[2 * s + 1 <= W ? 2 * s + 1 : 0] : zero);
            f[0][2 * s] = __builtin_bit_cast(u4, x.hi);
            f[0][2 * s + 1] = __builtin_bit_cast(u4, x.lo);
          }
          if (2 * s + 1 >= W) {
            const Parts x = parts(2 * s >= W ? upper[2 * s >= W ? 2 * s - W : 0] : zero, upper[2 * s + 1 >= W ? 2 * s + 1 - W : 0]);
            f[1][2 * s] = __builtin_bit_cast(u4, x.hi);
            f[1][2 * s + 1] = __builtin_bit_cast(u4, x.lo);
          }
        }
      };
      if constexpr (NW == 8) {
        if (w < 4) by_wave(w, [&](auto wave) { products(wave, std::false_type{}, frag[0]); });
        else by_wave(w - 4, [&](auto wave) { products(wave, std::true_type{}, frag[0]); });
      } else {
        by_wave(w, [&](auto wave) {
          products(wave, std::false_type{}, frag[0]);
          products(wave, std::true_type{}, frag[NW == 8 ? 0 : 1]);
        });
      }
      // Products over the values, 32 at a time, a wavefront per 16 key elements.
      f4v aq[4] = {}, ae[4] = {}, aw[4] = {};
      float both = 0.0f;
      const unsigned slice = base + kAtS;
#pragma unroll 1
      for (int s = 0; s < NV; ++s) {
        typedef __attribute__((address_space(3))) u2 lds8;
        const Parts sp = parts(sv[0], sv[1]), dp = parts(dv[0], dv[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int id4 = k * NT + tid, r = id4 / (KD / 4), e4 = id4 % (KD / 4);
          const unsigned to = slice + static_cast<unsigned>(slot<KD>(r, e4 >> 1)) * 16 + (e4 & 1) * 8;
          *(lds8 *)(to) = half_of(sp.hi, k);
          *(lds8 *)(to + kSlice) = half_of(sp.lo, k);
          *(lds8 *)(to + 2 * kSlice) = half_of(dp.hi, k);
          *(lds8 *)(to + 3 * kSlice) = half_of(dp.lo, k);
#pragma unroll
          for (int e = 0; e < 4; ++e) both = fmaf(sv[k][e], dv[k][e], both);
        }
        if (s + 1 < NV) fetch_slice(s + 1);
        meet();
        Parts so, dso;
        so = {values16<KD>(slice + col_s), values16<KD>(slice + kSlice + col_s)};
        dso = {values16<KD>(slice + 2 * kSlice + col_s), values16<KD>(slice + 3 * kSlice + col_s)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          aq[i] = mul_exact(row16<VD>(base + kAtD, i, s, atv), so, aq[i]);
          ae[i] = mul_parts(tokens16(D, i, s, col), so, ae[i]);
          aw[i] = mul_parts(tokens16(U, i, s, col), dso, aw[i]);
        }
        meet();
      }
      // Fragments of kind k take the place of U and D: as they are at 2 k, transposed at 2 k + 1.
      auto keep = [&](int W, int kind, const u4 (&f)[2][4]) {
        u4 *to = lds + (kAtU + kind * 2 * kGdrTriBytes) / 16 + lane;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (2 * s <= W) {
            to[tri(W, s) * 64] = f[0][2 * s];
            to[(kGdrFrags + tri(W, s)) * 64] = f[0][2 * s + 1];
          }
          if (2 * s + 1 >= W) {
            to[kGdrTriBytes / 16 + tri_t(W, s) * 64] = f[1][2 * s];
            to[kGdrTriBytes / 16 + (kGdrFrags + tri_t(W, s)) * 64] = f[1][2 * s + 1];
          }
        }
      };
      if constexpr (NW == 8) {
        keep(w & 3, w >> 2, frag[0]);
      } else {
        keep(w, 0, frag[0]);
        keep(w, 1, frag[NW == 8 ? 0 : 1]);
      }
      both *= gates[64 + 63];
      sh4 kc[4], qc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kc[i] = rows4<KD>(base, i, w, lane);
        qc[i] = rows4<KD>(base + kAtQ, i, w, lane);
        const f4v qs = *reinterpret_cast<const f4v *>(gates + 16 * i + 4 * g);
        const f4v into = *reinterpret_cast<const f4v *>(gates + 64 + 16 * i + 4 * g);
        const f4v out = *reinterpret_cast<const f4v *>(gates + 128 + 16 * i + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          aq[i][r] *= qs[r];
          ae[i][r] *= -into[r];
          aw[i][r] *= out[r];
          both = fmaf(up(kc[i][r]), aw[i][r], both);  // <S_C, dS> with what the chunk adds to S_C
        }
      }
      meet();
      const unsigned fp = base + kAtU, fh = fp + 2 * kGdrTriBytes;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bf8 kb = elems16<KD>(base, w, s, lane), qb = elems16<KD>(base + kAtQ, w, s, lane);
        auto mul = [&](unsigned f, int k, bf8 x, f4v acc) {
          return mfma16(frag16(f, k, lane), x, mfma16(frag16(f, kGdrFrags + k, lane), x, acc));
        };
#pragma unroll
        for (int i = 2 * s; i < 4; ++i) {
          aq[i] = mul(fp, tri(i, s), kb, aq[i]);
          ae[i] = mul(fh, tri(i, s), kb, ae[i]);
        }
#pragma unroll
        for (int j = 0; j <= 2 * s + 1; ++j) {
          aw[j] = mul(fp + kGdrTriBytes, tri_t(j, s), qb, aw[j]);
          aw[j] = mul(fh + kGdrTriBytes, tri_t(j, s), kb, aw[j]);
        }
      }
      // d / dG, a term per token from each of q, the key that reads and the key that writes.
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v = sum16(fmaf(up(qc[i][r]), aq[i][r], up(kc[i][r]) * (ae[i][r] - aw[i][r])));
          if (m == 0) red[1][w][16 * i + 4 * g + r] = v;
        }
        tq[i] += aq[i];
        tk[i] += ae[i] + aw[i];
      }
      both = sum16(both);
      both += __shfl_xor(both, 16);
      both += __shfl_xor(both, 32);
      if (lane == 0) whole[w] = both;
      meet();
      if (w == 0 && lane < rows) {
        float dg = 0.0f, dbeta = 0.0f, total = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          dbeta += red[0][k][lane];
          dg += red[1][k][lane];
          total += whole[k];
        }
        if (lane >= len) dg = dbeta = 0.0f;
        if (lane == (len < 64 ? len - 1 : 63)) dg += total;
        red[1][0][lane] = dg;
        store_gate(p.dbeta, (b * p.seqlen + t0 + lane) * p.nheads + h, dbeta, G{});
      }
      if (w == 0) {  // dg_t is the sum of d / dG from t on
        float v = lane < rows ? red[1][0][lane] : 0.0f;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const float next = __shfl_down(v, d);
          if (lane + d < 64) v += next;
        }
        if (lane < rows) store_gate(p.dg, (b * p.seqlen + t0 + lane) * p.nheads + h, lane < len ? v : 0.0f, G{});
      }
    }
  } else {
    for (int64_t i = threadIdx.x; i < rows * share; i += NT) {
      const int64_t to = (b * p.seqlen + t0 + i / share) * p.nheads + hk * share + i % share;
      store_gate(p.dg, to, 0.0f, G{});
      store_gate(p.dbeta, to, 0.0f, G{});
    }
  }
  const int m = threadIdx.x & 15, g = threadIdx.x >> 4 & 3;
  uint16_t *dqp = p.dq + ((b * p.seqlen + t0) * p.nqk + hk) * KD + 16 * w + m;
  uint16_t *dkp = p.dk + ((b * p.seqlen + t0) * p.nqk + hk) * KD + 16 * w + m;
  const int64_t row_step = p.nqk * KD;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * i + 4 * g + r;
      if (row < rows) {
        st(dqp, row * row_step, row < len ? tq[i][r] : 0.0f);
        st(dkp, row * row_step, row < len ? tk[i][r] : 0.0f);
      }
    }
}

template <int KD, int VD, typename G>
void grad(const GdrParams &p, hipStream_t s) {
  hipLaunchKernelGGL((gdr_grad_kernel<KD, VD, G>), dim3(static_cast<uint32_t>(p.batch * p.nqk * p.chunks)), dim3(4 * KD), 0, s, p);
}

template <int KD>
hipError_t bwd(const GdrParams &p, hipStream_t s) {
  const int64_t heads = p.batch * p.nheads;
  hipLaunchKernelGGL((gdr_bwd_kernel<KD>), dim3(static_cast<uint32_t>(heads * (p.vdim / 32))), dim3(256), 0, s, p);
  if (p.chunks > 0) {
    if (p.vdim == 64) p.gates_bf16 ? grad<KD, 64, uint16_t>(p, s) : grad<KD, 64, float>(p, s);
    else p.gates_bf16 ? grad<KD, 128, uint16_t>(p, s) : grad<KD, 128, float>(p, s);
  }
  return hipGetLastError();
}

}  // namespace

GdrBwdSizes gdr_bwd_sizes(const GdrParams &p) {
  const size_t n = static_cast<size_t>(p.batch) * p.nheads * p.chunks;
  return {n * kGdrBwdChunkBytes, n * p.vdim * p.kdim * 4, n * 64 * p.vdim * 4};
}

hipError_t launch_gdr_bwd(const GdrParams &p, hipStream_t s) {
  const hipError_t e = launch_gdr_chunks(p, true, s);
  if (e != hipSuccess) return e;
  return p.kdim == 64 ? bwd<64>(p, s) : bwd<128>(p, s);
}

}  // namespace ssmb
