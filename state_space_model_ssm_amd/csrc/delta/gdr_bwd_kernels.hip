// Gated delta rule, backward, for gfx950.
//
// With the forward's T, A, Z and states, dS the gradient of the state behind a
// chunk, and M_ij = e^(G_i - G_j):
//   D = T^T (A^T dY + beta e^(G_64 - G) K dS^T) = dV
//   dS' = e^(G_64) dS + (scale e^G dY)^T Q - (e^G D)^T K
//   P = scale (dY Z^T) M (j <= i),  H = -(D Z^T) M (j < i)
//   dQ = scale e^G dY S + (P beta) K
//   dK = (H beta) K - e^G D S + beta (e^(G_64 - G) Z dS + P^T Q + H^T K), as read and as written
// (beta by rows of the last sum and by columns of P and H in the others).  With
//   W_ij = P_ij q_i.k_j + H_ij k_i.k_j,  c_j = k_j.(e^(G_64 - G) Z dS)_j
// dbeta_j is D_j.Z_j / beta_j, or, where beta is 0, c_j and the sum of W over
// i >= j (the same; but keys that are alike make that sum's terms cancel: 4e-5
// off by norms, not 1e-5),
// and dg_t is the sum of the terms whose decay passes token t, those of
//   W_ij beta_j   from j < t to i >= t
//   q_i.(scale e^G dY S)_i - k_i.(e^G D S)_i   for i >= t, from the state before
//   c_j beta_j   for j < t, to the state behind, and e^(G_64) <S, dS>
// each of which has a_t as a factor, as dg_t itself does.  (The sum over i >= t
// of what G_i's gradient is, q_i.dq_i + k_i.(dk_i as read - dk_i as written),
// is the same without W; but all that lies behind t has to cancel in it then,
// and where a_t is small only the roundings of that are left.)
//
// A first kernel goes from chunk to chunk backwards with dS (as the forward,
// bound by its chain; 3.4 us a chunk with the 96 KiB of dS and D that it leaves
// behind), and is cut into segments where heads are few; a second has all
// chunks at once and is bound by reading those and what the forward saved.
// Roundings: q, k and dy are exact; S, Z, dS, D, T, A, P and H enter products as
// two bfloat16 parts, 2^-18 of their size, and products of two such leave out the
// smallest term; sums are float32.  So dg, dbeta and dh0, which are stored in
// float32 where the gates are (dh0 always), are 2e-6 to 1.2e-5 off by norms,
// where float32 token by token is 2e-7 to 2e-6.  They are linear in dy and
// dh_last: dy's own rounding to bfloat16 has left 2^-9 a value in them, 150 times
// more.  Three parts, as the forward's last state has, would take half as many
// bytes again of what it saves and what these kernels hand on, which bound them.
//
// Measured, 4 x 2048 tokens, 16 heads of 128: 109 us, and 157 for 557 MB (3.5
// TB/s, where a large read reaches 4.0); a training pass 375 us with the
// forward.  With keys of 128 the second kernel has more than its 256 registers:
// 13 are spilled, 125 to 130 where value heads share keys, whose sums it carries
// along (8 query heads: 378 us all the same).
#include "gdr_tile.h"

namespace ssmb {
namespace {

// ---------------------------------------------------------------------------
// From chunk to chunk, the last one first: dS, and D = dv
// ---------------------------------------------------------------------------

// As in the forward two wavefronts carry dS, 16 columns each, and two others
// make what does not depend on it, A^T dY and Q^T (scale e^G dY), copy the next
// chunk, and store D and dv.  FIND: of all segments but the first, only the dS
// before it, from 0 or, of a row's last, from dh_last.
template <int KD, bool FIND>
__global__ void __launch_bounds__(256) gdr_bwd_kernel(const GdrParams p) {
  constexpr int NT = 64 * kPairs, NC = 16 * kPairs, NS = KD / 32, NB = KD / 16;
  constexpr unsigned kRows = 64 * KD * 2, kValues = 64 * NC * 2, kTri = 2 * kGdrTriBytes, kOps = kTri + kGdrGateBytes;
  constexpr unsigned kAtQ = kRows, kAtD = 2 * kRows, kAtW = kAtD + kValues, kBuffer = kAtW + kOps;
  constexpr unsigned kFour = 4 * 1024, kState = NB * 1024;  // D results of the tokens and of the state: float32, or two parts
  __shared__ __align__(16) u4 lds[(2 * kBuffer + kPairs * (kFour + kState)) / 16];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave % kPairs;
  const unsigned vtiles = static_cast<unsigned>(p.vdim) / NC;
  const HeadTile which = head_tile(blockIdx.x, static_cast<unsigned>(p.batch * p.nheads), vtiles * static_cast<unsigned>(p.seg.count - (FIND ? 1 : 0)));
  const int64_t vt = which.tile % vtiles, bh = which.head, b = bh / p.nheads, h = bh % p.nheads;
  // Chunks n - 1 .. first of the row, of this segment.
  const int segment = static_cast<int>(which.tile / vtiles) + (FIND ? 1 : 0), len = gdr_length(p.lengths, b, p.seqlen);
  const int first = segment * static_cast<int>(p.seg.chunks), all = (len + 63) / 64;
  const int n = all < first + p.seg.chunks ? all : first + static_cast<int>(p.seg.chunks);
  if (FIND && n <= first) return;
  const int col0 = static_cast<int>(vt) * NC + 16 * w;
  const unsigned base = lds_at(lds), four = base + 2 * kBuffer + w * kFour + lane * 16;
  const unsigned grown = base + 2 * kBuffer + kPairs * kFour + w * kState + lane * 16;
  const Lanes16 at = lanes16_of<KD>(lane);
  typedef __attribute__((address_space(3))) f4v lds_f4v;
  typedef __attribute__((address_space(3))) u4 lds16;

  if (wave < kPairs) {
    f4v s[NB];  // dS, laid out as the state
    const int64_t state = (bh * p.vdim + col0 + m) * KD + 8 * g;
    float *behind = p.ws_state + ((bh * p.seg.count + segment) * p.vdim + col0 + m) * KD + 8 * g;
    const float *from = first + p.seg.chunks >= all ? (p.dh_last != nullptr ? p.dh_last + state : nullptr) : FIND ? nullptr : behind;
#pragma unroll
    for (int j = 0; j < NB; ++j)
      s[j] = from != nullptr ? *reinterpret_cast<const f4v *>(from + 32 * (j / 2) + 4 * (j % 2)) : f4v{};
    for (int c = n - 1; c >= first; --c) {
      Parts sp[NS];
#pragma unroll
      for (int a = 0; a < NS; ++a) {
        sp[a] = parts(s[2 * a], s[2 * a + 1]);
        *(lds16 *)(grown + a * 2048) = __builtin_bit_cast(u4, sp[a].hi);
        *(lds16 *)(grown + a * 2048 + 1024) = __builtin_bit_cast(u4, sp[a].lo);
      }
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
        fac[i] = -lds_f4(gates + 256 + 64 * i);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j <= 2 * k + 1; ++j) tf[tri_t(j, k)] = {tri_cols(at_t, j, k, 0, lane), tri_cols(at_t, j, k, 1, lane)};
      const float whole = lds_f4(at_t + kTri + 256 + 240)[3];
      __builtin_amdgcn_sched_barrier(0);
      // K dS, and beta e^(GC - G) of that + A^T dY
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
      // D = T^T of that
      f4v e[4] = {x[0], x[1], x[2], x[3]};
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
      // dS = e^GC dS + sum over tokens of q (scale e^G dy) - k (e^G D)
#pragma unroll
      for (int j = 0; j < NB; ++j) s[j] = s[j] * whole + *(const lds_f4v *)(grown + j * 1024);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NB; ++j) s[j] = mul_exact(kt[k][j], ep[k], s[j]);
    }
    float *to = FIND ? behind - p.vdim * KD : segment == 0 && p.dh0 != nullptr ? p.dh0 + state : nullptr;
    if (to != nullptr) {
#pragma unroll
      for (int j = 0; j < NB; ++j) *reinterpret_cast<f4v *>(to + 32 * (j / 2) + 4 * (j % 2)) = s[j];
    }
    return;
  }

  const int id = tid - NT;
  const int64_t hk = h / (p.nheads / p.nqk), yt = p.nheads * p.vdim;
  const uint16_t *kp = p.k + b * p.k_batch + hk * KD, *qp = p.q + b * p.q_batch + hk * KD;
  const uint16_t *dp = p.dy + (b * p.seqlen * p.nheads + h) * p.vdim + vt * NC;
  const int64_t step = static_cast<int64_t>(gdr_saved_bytes(KD, p.vdim));
  const char *ws = p.saved + bh * p.chunks * step + gdr_both_bytes(KD, p.vdim);  // T, A, gates
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
    copy_share<kOps / 1024, kPairs>(base + (c & 1) * kBuffer + kAtW, ws + c * step, w, lane * 16);
  };
  f4v e[4];
  const int64_t nv = p.vdim / 32;
  auto both = [&](int c) {
    return p.ws_both + (bh * p.chunks + c) * static_cast<int64_t>(gdr_both_bytes(KD, p.vdim)) + lane * 16;
  };
  // D: dv, and operands over the values, of which this column tile has halves.
  sh4 dt[4][2];
  auto turn = [&](int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = *(const lds_f4v *)(four + i * 1024);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Parts d = parts(e[2 * k], e[2 * k + 1]);
      *(lds16 *)(four + k * 2048) = __builtin_bit_cast(u4, d.hi);
      *(lds16 *)(four + k * 2048 + 1024) = __builtin_bit_cast(u4, d.lo);
    }
    wait_reads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int part = 0; part < 2; ++part) dt[i][part] = turned<false>(four - lane * 16, i, part, lane);
    if (64 * c + 64 > len) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (64 * c + 16 * i + 4 * g + r >= len) e[i][r] = 0.0f;
    }
  };
  auto store = [&](int c) {
    char *to = both(c) + gdr_state_bytes(KD, p.vdim) + vt * 8192 + w * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int part = 0; part < 2; ++part) __builtin_nontemporal_store(dt[i][part], reinterpret_cast<sh4 *>(to + i * 2048 + part * 1024));
    const int64_t rest = p.seqlen - 64 * static_cast<int64_t>(c);
    v_store.put(vp + 64 * c * yt, rest < 64 ? static_cast<int>(rest) : 64, e);
  };
  if (n > first) {
    fetch_rows(n - 1);
    fetch_ws(n - 1);
  }
  for (int c = n - 1; c >= first; --c) {
    arrive();
    if (!FIND && c + 1 < n) store(c + 1);
    // dS behind the chunk, half of both columns' tiles by each of the two wavefronts.
    const unsigned all_s = base + 2 * kBuffer + kPairs * kFour;
    char *to = both(c) + vt * 2048;
#pragma unroll
    for (int j = 0; j < (FIND ? 0 : NB / 2); ++j)
#pragma unroll
      for (int part = 0; part < 2; ++part)
        __builtin_nontemporal_store(turned<true>(all_s, all_s + kState, 2 * j + w, part, lane),
                                    reinterpret_cast<bf8 *>(to + (2 * j + w) * nv * 2048 + part * 1024));
    const unsigned tile = base + (c & 1) * kBuffer, at_a = tile + kAtW + kGdrTriBytes, gates = at_a + kGdrTriBytes + 16 * g;
    Parts af[kGdrFrags];
    sh4 dy[4];
    bf8 qt[2][NB];
#pragma unroll
    for (int i = 0; i < 4; ++i) dy[i] = rows4<NC>(tile + kAtD, i, w, lane);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j <= 2 * k + 1; ++j) af[tri_t(j, k)] = {tri_cols(at_a, j, k, 0, lane), tri_cols(at_a, j, k, 1, lane)};
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
    if (c > first) fetch_rows(c - 1);
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
    if (c > first) fetch_ws(c - 1);
    if (!FIND) turn(c);
  }
  if (FIND) return;
  if (n > first) store(first);
  const int64_t last = segment + 1 < p.seg.count ? 64 * (first + p.seg.chunks) : p.seqlen;  // the segment's rows behind the length
  for (int64_t row = 64 * static_cast<int64_t>(n > first ? n : first) + g; row < last && row < p.seqlen; row += 4) st(vp, row * yt + m, 0.0f);
}

// ---------------------------------------------------------------------------
// Within a chunk: dq, dk, dg, dbeta
// ---------------------------------------------------------------------------

// The sum over the 16 lanes of a row.
__device__ __forceinline__ float sum16(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true));
  return v;
}

// The sum over the lanes before.
__device__ __forceinline__ float sum_before(float v) {
  v = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x138, 0xf, 0xf, false));   // from the lane before
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xf, 0xf, false));  // 1, 2, 4, 8 before, of 16
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xf, 0xf, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xf, 0xf, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xf, 0xf, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xa, 0xf, false));  // the last of the 16 before
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xc, 0xf, false));  // and of the 32
  return v;
}

__device__ __forceinline__ void store_gate(void *p, int64_t i, float v, float) { st(static_cast<float *>(p), i, v); }
__device__ __forceinline__ void store_gate(void *p, int64_t i, float v, uint16_t) { st(static_cast<uint16_t *>(p), i, v); }

// A fragment of 1024 bytes in memory.  (Read once: past the caches, which hold
// what the head's other wavefronts read; 169 -> 160 us with 2048 chunks of 128.)
__device__ __forceinline__ bf8 frag_at(const char *p, int lane) {
  return __builtin_nontemporal_load(reinterpret_cast<const bf8 *>(p + lane * 16));
}

// Operand of rows 16 i .. of a tile of 64 values a row, k its values 32 s .. in D's order.
__device__ __forceinline__ bf8 row16_d(unsigned tile, int i, int s, unsigned row) {
  typedef __attribute__((address_space(3))) const u2 lds8;
  const unsigned at = ((tile + row) ^ (64 * s)) + i * 2048;
  const u2 lo = *(lds8 *)(at), hi = *(lds8 *)(at ^ 32);
  return __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3));
}

__device__ __forceinline__ float dot2(bf8 a, bf8 b, float c) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf2;
#pragma unroll
  for (int k = 0; k < 4; ++k) c = __builtin_amdgcn_fdot2_f32_bf16(bf2{a[2 * k], a[2 * k + 1]}, bf2{b[2 * k], b[2 * k + 1]}, c, false);
  return c;
}

// A workgroup per chunk and query head, over the value heads that share it; a
// wavefront per quarter of the key elements, and per 16 tokens of what the
// tokens are to each other.
template <int KD, int VD, bool SHARED, typename G>
__global__ void __launch_bounds__(256, 2) gdr_grad_kernel(const GdrParams p) {
  constexpr int NT = 256, NW = 4, NE = KD / 64, NV = VD / 32;  // NE: blocks of 16 key elements of a wavefront
  constexpr unsigned kRows = 64 * KD * 2, kAtQ = kRows, kAtD = 2 * kRows, kAtU = kAtD + 64 * 64 * 2, kParts = 2 * 8 * 1024;
  // dY, Z and D of 64 values; then fragments of a triangle and its transpose, and the triangle in float32.
  constexpr unsigned kTriangle = 2 * kGdrTriBytes, kValues = 64 * 64 * 2 + 2 * kParts, kAll = kTriangle + 64 * kPitch * 4;
  constexpr unsigned kArea = kValues > kAll ? kValues : kAll;
  __shared__ __align__(16) u4 lds[(kAtD + kArea) / 16];
  __shared__ float red[4][NW][64], diag[64], whole[NW];  // red: sums of W for dg and for dbeta, and the tokens' terms with S and with dS
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned chunks = static_cast<unsigned>(p.chunks), nqk = static_cast<unsigned>(p.nqk);
  const int64_t c = blockIdx.x % chunks, bk = blockIdx.x / chunks, b = static_cast<unsigned>(bk) / nqk, hk = static_cast<unsigned>(bk) % nqk;
  const int64_t share = static_cast<unsigned>(p.nheads) / nqk;
  const int t0 = static_cast<int>(c) * 64, len = gdr_length(p.lengths, b, p.seqlen) - t0;
  const int rows = p.seqlen - t0 < 64 ? static_cast<int>(p.seqlen - t0) : 64;
  f4v aq[NE][4] = {}, ak[NE][4] = {};  // dq and dk
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
      const unsigned row = static_cast<unsigned>(slot<64>(m, g >> 1)) * 16 + (g & 1) * 8;
      const int64_t bh = b * p.nheads + h, id = bh * p.chunks + c, yt = p.nheads * VD;
      const char *fs = p.saved + id * static_cast<int64_t>(gdr_saved_bytes(KD, VD)), *fu = fs + gdr_state_bytes(KD, VD);
      const char *fds = p.ws_both + id * static_cast<int64_t>(gdr_both_bytes(KD, VD)), *fd = fds + gdr_state_bytes(KD, VD);
      const float *gates = reinterpret_cast<const float *>(fs + gdr_both_bytes(KD, VD) + 2 * kGdrTriBytes);
      const double *sums = reinterpret_cast<const double *>(gates + 256);
      const uint16_t *dyp = p.dy + (b * p.seqlen * p.nheads + h) * VD;
      f4v tq[NE][4], tk[NE][4];  // of the heads before
      if (SHARED)
#pragma unroll
        for (int x = 0; x < NE; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tq[x][i] = aq[x][i];
            tk[x][i] = ak[x][i];
            aq[x][i] = f4v{};
          }
      f4v ae[NE][4] = {}, aw[NE][4] = {};  // what keys get as they read, and as they write
      f4v py[4] = {}, pd[4] = {};          // dY Z^T and D Z^T: rows j, columns i = 16 w + m
      float both = 0.0f;
#pragma unroll 1
      for (int hv = 0; hv < VD / 64; ++hv) {
        arrive();  // what was in LDS has been read
        load_tile<64, NT>(lds + kAtD / 16, dyp + 64 * hv, yt, t0, t0 + len - 1, tid);
        copy_share<16, NW>(base + kAtU, fu + hv * 16384, w, lane * 16);
        copy_share<16, NW>(base + kAtU + kParts, fd + hv * 16384, w, lane * 16);
        Parts sp[NE], dp[NE];
        auto load = [&](int s) {
#pragma unroll
          for (int x = 0; x < NE; ++x) {
            const int64_t at = ((NE * w + x) * NV + 2 * hv + s) * 2048;
            sp[x] = {frag_at(fs + at, lane), frag_at(fs + at + 1024, lane)};
            dp[x] = {frag_at(fds + at, lane), frag_at(fds + at + 1024, lane)};
          }
        };
        load(0);
        arrive();
        const unsigned dy = base + kAtD, u = base + kAtU, d = u + kParts;
        auto part = [&](unsigned from, int i, int s) {  // Z or D, token block i
          return Parts{frag16(from, (4 * s + i) * 2, lane), frag16(from, (4 * s + i) * 2 + 1, lane)};
        };
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          const Parts dw = part(d, w, s);
          const bf8 yw = row16_d(dy, w, s, row);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Parts ui = part(u, i, s), di = part(d, i, s);
            const bf8 yi = row16_d(dy, i, s, row);
            py[i] = mfma16(ui.hi, yw, mfma16(ui.lo, yw, py[i]));
            pd[i] = mul_parts(ui, dw, pd[i]);
#pragma unroll
            for (int x = 0; x < NE; ++x) {
              aq[x][i] = mul_exact(yi, sp[x], aq[x][i]);
              ae[x][i] = mul_parts(di, sp[x], ae[x][i]);
              aw[x][i] = mul_parts(ui, dp[x], aw[x][i]);
            }
          }
#pragma unroll
          for (int x = 0; x < NE; ++x) both = dot2(sp[x].hi, dp[x].hi, dot2(sp[x].hi, dp[x].lo, dot2(sp[x].lo, dp[x].hi, both)));
          if (s == 0) load(1);
        }
      }
      meet();  // what was in LDS has been read
      // P = scale (dY Z^T) M, H = -(D Z^T) M and W, and the diagonal of D Z^T.
      const int own = 16 * w + m;
      const double so = sums[own];
      const Lanes16 at = lanes16_of<KD>(lane);
      float *full = reinterpret_cast<float *>(lds + kAtD / 16 + kTriangle / 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f4v qk = {}, kk = {};  // q_i.k_j and k_i.k_j, laid out as P and H
#pragma unroll
        for (int a = 0; a < KD / 32; ++a) {
          const bf8 kj = row16<KD>(base, j, a, at);
          qk = mfma16(kj, row16<KD>(base + kAtQ, w, a, at), qk);
          kk = mfma16(kj, row16<KD>(base, w, a, at), kk);
        }
        f4v sum;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int other = 16 * j + 4 * g + r;
          const float gap = static_cast<float>(so - sums[other]);
          if (other == own) diag[own] = pd[j][r];
          const float decay = __builtin_amdgcn_exp2f(gap);
          py[j][r] = other <= own && own < len ? py[j][r] * p.scale * decay : 0.0f;
          pd[j][r] = other < own ? -pd[j][r] * decay : 0.0f;
          sum[r] = fmaf(py[j][r], qk[r], pd[j][r] * kk[r]);
        }
        *reinterpret_cast<f4v *>(full + own * kPitch + 16 * j + 4 * g) = sum;
      }
      wait_reads();
      {  // Lane t: W beta from j < t to this wavefront's i >= t, and W from j = t.
        const float beta = gates[192 + lane];
        float cut = 0.0f, column = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float here = full[(16 * w + i) * kPitch + lane], before = sum_before(here * beta);
          cut += 16 * w + i >= lane ? before : 0.0f;
          column += here;
        }
        red[0][w][lane] = cut;
        red[3][w][lane] = column;
      }
      both *= gates[64 + 63];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f4v qs = *reinterpret_cast<const f4v *>(gates + 16 * i + 4 * g);
        const f4v into = *reinterpret_cast<const f4v *>(gates + 64 + 16 * i + 4 * g);
        const f4v out = *reinterpret_cast<const f4v *>(gates + 384 + 16 * i + 4 * g);
        f4v before = {}, behind = {};
#pragma unroll
        for (int x = 0; x < NE; ++x) {
          const sh4 kc = rows4<KD>(base, i, NE * w + x, lane), qc = rows4<KD>(base + kAtQ, i, NE * w + x, lane);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            aq[x][i][r] *= qs[r];
            ae[x][i][r] *= -into[r];
            aw[x][i][r] *= out[r];
            before[r] = fmaf(up(qc[r]), aq[x][i][r], fmaf(up(kc[r]), ae[x][i][r], before[r]));
            behind[r] = fmaf(up(kc[r]), aw[x][i][r], behind[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float b0 = sum16(before[r]), b1 = sum16(behind[r]);
          if (m == 0) {
            red[1][w][16 * i + 4 * g + r] = b0;
            red[2][w][16 * i + 4 * g + r] = b1;
          }
        }
      }
      // P and P^T, then H and H^T, as fragments in LDS, where all wavefronts take them.
      const unsigned area = base + kAtD;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        meet();
        const f4v (&lower)[4] = kind == 0 ? py : pd;
        u4 *to = lds + kAtD / 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<f4v *>(full + own * kPitch + 16 * j + 4 * g) = lower[j];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const f4v *beta = reinterpret_cast<const f4v *>(gates + 192 + 32 * s + 4 * g);
          const Parts x = parts(lower[2 * s] * beta[0], lower[2 * s + 1] * beta[4]);
          if (2 * s <= w) {
            const int f = w < 2 ? w : 2 * (w - 1) + s;
            to[f * 64 + lane] = __builtin_bit_cast(u4, x.hi);
            to[(kGdrFrags + f) * 64 + lane] = __builtin_bit_cast(u4, x.lo);
          }
        }
        meet();
        store_cols(full, w, to + kGdrTriBytes / 16, lane);
        meet();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          bf8 kb[NE], qb[NE];
#pragma unroll
          for (int x = 0; x < NE; ++x) {
            kb[x] = elems16<KD>(base, NE * w + x, s, lane);
            if (kind == 0) qb[x] = elems16<KD>(base + kAtQ, NE * w + x, s, lane);
          }
#pragma unroll
          for (int i = 2 * s; i < 4; ++i) {
            const Parts f = {frag16(area, tri(i, s), lane), frag16(area, kGdrFrags + tri(i, s), lane)};
#pragma unroll
            for (int x = 0; x < NE; ++x) {
              f4v &acc = kind == 0 ? aq[x][i] : ae[x][i];
              acc = mfma16(f.hi, kb[x], mfma16(f.lo, kb[x], acc));
            }
          }
#pragma unroll
          for (int j = 0; j <= 2 * s + 1; ++j) {
            const Parts f = {frag16(area + kGdrTriBytes, tri_t(j, s), lane), frag16(area + kGdrTriBytes, kGdrFrags + tri_t(j, s), lane)};
#pragma unroll
            for (int x = 0; x < NE; ++x) {
              const bf8 right = kind == 0 ? qb[x] : kb[x];
              aw[x][j] = mfma16(f.hi, right, mfma16(f.lo, right, aw[x][j]));
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f4v beta = *reinterpret_cast<const f4v *>(gates + 192 + 16 * i + 4 * g);
#pragma unroll
        for (int x = 0; x < NE; ++x) {
          ak[x][i] = ae[x][i] + beta * aw[x][i];
          if (SHARED) {
            aq[x][i] += tq[x][i];
            ak[x][i] += tk[x][i];
          }
        }
      }
      both = sum16(both);
      both += __shfl_xor(both, 16);
      both += __shfl_xor(both, 32);
      if (lane == 0) whole[w] = both;
      meet();
      if (w == 0) {
        const float beta = gates[192 + lane];
        float dg = 0.0f, before = 0.0f, behind = 0.0f, dbeta = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          dg += red[0][k][lane] + whole[k];
          before += red[1][k][lane];
          behind += red[2][k][lane];
          dbeta += red[3][k][lane];
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const float next = __shfl_down(before, d);
          if (lane + d < 64) before += next;
        }
        dg += before + sum_before(beta * behind);
        dbeta = fabsf(beta) >= 0x1p-100f ? diag[lane] / beta : dbeta + behind;
        if (lane < rows) {
          const int64_t to = (b * p.seqlen + t0 + lane) * p.nheads + h;
          store_gate(p.dg, to, lane < len ? dg : 0.0f, G{});
          store_gate(p.dbeta, to, lane < len ? dbeta : 0.0f, G{});
        }
      }
    }
  } else {
    for (int64_t i = threadIdx.x; i < rows * share; i += NT) {
      const int64_t to = (b * p.seqlen + t0 + i / share) * p.nheads + hk * share + i % share;
      store_gate(p.dg, to, 0.0f, G{});
      store_gate(p.dbeta, to, 0.0f, G{});
    }
  }
  const int lane = threadIdx.x & 63, g = lane >> 4;
  RowStore out;
  out.init(p.nqk * KD, lane);
#pragma unroll
  for (int x = 0; x < NE; ++x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (16 * i + 4 * g + r >= len) aq[x][i][r] = ak[x][i][r] = 0.0f;
    const int64_t to = ((b * p.seqlen + t0) * p.nqk + hk) * KD + 16 * (NE * w + x);
    out.put(p.dq + to, rows, aq[x]);
    out.put(p.dk + to, rows, ak[x]);
  }
}

template <int KD, int VD, typename G>
void grad(const GdrParams &p, hipStream_t s) {
  const dim3 n(static_cast<uint32_t>(p.batch * p.nqk * p.chunks));
  if (p.nheads == p.nqk) hipLaunchKernelGGL((gdr_grad_kernel<KD, VD, false, G>), n, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((gdr_grad_kernel<KD, VD, true, G>), n, dim3(256), 0, s, p);
}

template <int KD>
hipError_t bwd(const GdrParams &p, hipStream_t s) {
  const int64_t heads = p.batch * p.nheads;
  const int64_t columns = heads * (p.vdim / 32);
  if (p.seg.count > 1) {
    hipLaunchKernelGGL((gdr_bwd_kernel<KD, true>), dim3(static_cast<uint32_t>(columns * (p.seg.count - 1))), dim3(256), 0, s, p);
    if (p.seg.count > 2) {
      launch_gdr_bwd_carry(p, s);
      launch_gdr_bwd_join(p, s);
    }
  }
  hipLaunchKernelGGL((gdr_bwd_kernel<KD, false>), dim3(static_cast<uint32_t>(columns * p.seg.count)), dim3(256), 0, s, p);
  if (p.chunks > 0) {
    if (p.vdim == 64) p.gates_bf16 ? grad<KD, 64, uint16_t>(p, s) : grad<KD, 64, float>(p, s);
    else p.gates_bf16 ? grad<KD, 128, uint16_t>(p, s) : grad<KD, 128, float>(p, s);
  }
  return hipGetLastError();
}

}  // namespace

GdrSegments gdr_bwd_segments(int64_t heads, int64_t kdim, int64_t vdim, int64_t chunks) {
  // As gdr_segments(): in turn a chunk takes 2.7 us (keys of 64: 1.9), without
  // what is stored 2.3 (1.7).  Forward and backward together, us a call: 2 heads
  // of 64, 8192 tokens: 1 segment of the backward 330, 8 169, 32 128; 8 of 128 on
  // 2, 2048 tokens: 1 222, 8 189, 16 203; 16 of 128, 4 x 2048: 1 368, 2 420.
  const bool wide = kdim == 128;
  const int64_t columns = heads * (vdim / 32), pairs = heads * (kdim / 64);
  int64_t best = 1;
  double least = (wide ? 2.7 : 1.9) * static_cast<double>(chunks) + 4.0;
  for (int64_t g = 2; g <= 64 && g <= chunks && columns * g <= 256; ++g) {
    const double each = static_cast<double>((chunks + g - 1) / g);
    double us = ((wide ? 2.3 : 1.7) + (wide ? 2.7 : 1.9)) * each + 8.0;
    if (g > 2) us += (wide ? 2.0 : 1.45) * each * static_cast<double>((pairs * (g - 2) + 255) / 256) + 8.0 + (wide ? 1.2 : 0.4) * static_cast<double>(g);
    if (us < least) {
      least = us;
      best = g;
    }
  }
  const int64_t each = (chunks + best - 1) / best;
  return {each > 0 ? (chunks + each - 1) / each : 1, each > 0 ? each : 1};
}

GdrSizes gdr_bwd_sizes(const GdrParams &p) {
  const size_t heads = static_cast<size_t>(p.batch) * p.nheads, n = p.seg.count > 1 ? heads * p.seg.count : 0;
  return {heads * p.chunks * gdr_both_bytes(p.kdim, p.vdim), 0, n * p.vdim * p.kdim * 4, n * 2 * p.kdim * p.kdim * 2};
}

hipError_t launch_gdr_bwd(const GdrParams &p, hipStream_t s) { return p.kdim == 64 ? bwd<64>(p, s) : bwd<128>(p, s); }

}  // namespace ssmb
