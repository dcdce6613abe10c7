// Gated delta rule, forward and single tokens, for gfx950.
//
// 64 tokens at a time.  With G_t the sum of g from the chunk's start to t, K, Q,
// V its tokens as rows and S the state before it (value elements x key
// elements), the z_t = u_t / beta_t of the tokens solve a triangular system:
//   L_ij = e^(G_i - G_j) k_i.k_j beta_j (j < i),  T = (I + L)^-1
//   Z = T (V - e^G K S^T)
//   A_ij = scale e^(G_i - G_j) q_i.k_j beta_j (j <= i),  Y = scale e^G Q S^T + A Z
//   S' = e^(G_64) S + (beta e^(G_64 - G) Z)^T K
// beta stands with what a token writes, so that a token whose beta is 0 leaves
// all others as they are, and its own z is there for beta's gradient.
// Exponents are differences that are at most 0 where g is: nothing overflows,
// and a strong decay is a 0.  T and A need no state: a first kernel makes them
// for all chunks at once.  What is left is a chain from chunk to chunk of three
// products, whose latency bounds the forward, not its arithmetic (14 to 20% of
// the matrix cores' time) nor its bytes: each value column's chain is its own, so
// the columns are spread over all compute units, and where they do not fill
// them, time is cut into segments (see gdr_segments()).
//
// Rounding: keys, queries and values are exact; T - I, A and what of S and Z
// makes y and is saved enter products as two bfloat16 parts, to 2^-18 of their
// size.  Two would leave the state itself 4e-6 off at the end, by norms, where
// float32 token by token is 2e-7 to 1e-6: where it is returned, S, Z, T - I and
// what T takes are in three parts as they make the next S (2^-26; 2.5e-7 to
// 8e-7 off with the rest), and so are a segment's E and P.  (T - I in two: 7e-7
// with random keys, 2e-6 to 6e-6 with keys that are alike.)  That costs a
// quarter of the chain's time (16 heads of 128, 8192 tokens: 199 us, 151
// without).  T's ones are kept out of what is rounded.  Sums are float32, sums of
// g float64.
//
// Measured, 16 heads of 128: one prompt of 8192 tokens in 199 us a call (chunks
// 31 us, segments 82, join 15, y 96); training's 4 x 2048, where the last state
// is not asked for, in 31 and 103, of which saving for the backward, 200 MB, is
// a third.
#include "gdr_tile.h"

namespace ssmb {
namespace {

// ---------------------------------------------------------------------------
// Within a chunk
// ---------------------------------------------------------------------------

constexpr int kDiagPitch = 20;  // floats between rows in LDS

// Store row block W of a lower triangle, transposed D results, as fragments in
// two parts, and the third where there is a place for it.
template <int W>
__device__ __forceinline__ void store_rows(const f4v (&t)[W + 1], u4 *to, u4 *rest, int lane) {
#pragma unroll
  for (int s = 0; 2 * s <= W; ++s) {
    const Parts3 x = parts3(t[2 * s], 2 * s + 1 <= W ? t[2 * s + 1 <= W ? 2 * s + 1 : 0] : f4v{});
    to[tri(W, s) * 64 + lane] = __builtin_bit_cast(u4, x.hi);
    to[(kGdrFrags + tri(W, s)) * 64 + lane] = __builtin_bit_cast(u4, x.lo);
    if (rest != nullptr) rest[tri(W, s) * 64 + lane] = __builtin_bit_cast(u4, x.rest);
  }
}
// The third parts, from memory: in the order of fragments.
__device__ __forceinline__ void load_rest(bf8 (&t)[kGdrFrags], const char *from, int lane) {
#pragma unroll
  for (int f = 0; f < kGdrFrags; ++f) t[f] = *reinterpret_cast<const bf8 *>(from + f * 1024 + lane * 16);
}

// One workgroup per chunk and value head, one wavefront per 16 of its tokens.
// T by blocks of 16: those on the diagonal by substitution, the others from
// them by products in float32, since errors of T's entries would grow along its
// rows.  2048 chunks of 128 in 31 us, where their 121 MB would take 25.  (Keys
// through LDS, not from memory by each wavefront: 37.)
template <int KD, typename G>
__global__ void __launch_bounds__(256) gdr_chunk_kernel(const GdrParams p) {
  // Keys, and after their products L^T and (the blocks of T on the diagonal)^T.
  constexpr int kTiles = 64 * KD * 2, kAfter = (64 * kPitch + 64 * kDiagPitch) * 4;
  __shared__ __align__(16) u4 lds[(kTiles > kAfter ? kTiles : kAfter) / 16];
  __shared__ double all_sums[4][64];  // log2 of the decay up to each token, of each wavefront
  __shared__ float all_betas[4][64];
  float *low = reinterpret_cast<float *>(lds), *diag = low + 64 * kPitch;
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t id = blockIdx.x, c = id % p.chunks, bh = id / p.chunks, b = bh / p.nheads, h = bh % p.nheads;
  const int t0 = static_cast<int>(c) * 64, len = gdr_length(p.lengths, b, p.seqlen) - t0;
  if (len <= 0) return;
  char *ws = p.ops + id * p.ops_step;
  constexpr int NS = KD / 32;
  const int64_t hk = h / (p.nheads / p.nqk);
  const int i = 16 * w + m, last_row = t0 + (len < 64 ? len : 64) - 1;  // rows past the length repeat the last one
  load_tile<KD, 256>(lds, uniform(p.k + b * p.k_batch + t0 * p.k_token + hk * KD), p.k_token, 0, last_row - t0, tid);
  // Queries, of which a wavefront takes its own only, straight to registers.
  bf8 qi[NS];
#pragma unroll
  for (int a = 0; a < NS; ++a)
    qi[a] = *reinterpret_cast<const bf8 *>(p.q + b * p.q_batch + (t0 + i < last_row ? t0 + i : last_row) * p.q_token + hk * KD + 32 * a + 8 * g);
  // Every wavefront makes the gates' sums for itself, while the keys and queries are on their way.
  double *sums = all_sums[w];
  float *betas = all_betas[w];
  {
    const int64_t from = (b * p.seqlen + t0 + (lane < len ? lane : len - 1)) * p.nheads + h;
    float gt = gate<G>(p.g, from), bt = gate<G>(p.beta, from);
    gt = gt < -200.0f ? -200.0f : gt;  // exp(-200) is 0, and differences of the sums stay finite
    if (lane >= len) gt = bt = 0.0f;  // nothing is added
    // In float64: after a strong decay the differences of later tokens' sums would lose what they have.
    double s = static_cast<double>(gt) * 1.4426950408889634;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double up = __shfl_up(s, d);
      if (lane >= d) s += up;
    }
    sums[lane] = s;
    betas[lane] = bt;
    const double last = __shfl(s, 63);
    if (w == 0) {
      const float into = __builtin_amdgcn_exp2f(static_cast<float>(s));
      float *gates = reinterpret_cast<float *>(ws + 2 * kGdrTriBytes);
      gates[lane] = lane < len ? p.scale * into : 0.0f;
      gates[64 + lane] = into;
      const float out = __builtin_amdgcn_exp2f(static_cast<float>(last - s));
      gates[128 + lane] = bt * out;
      gates[192 + lane] = bt;
      gates[384 + lane] = out;
      reinterpret_cast<double *>(gates + 256)[lane] = s;
    }
  }
  arrive();
  const unsigned keys = lds_at(lds);
  const Lanes16 at = lanes16_of<KD>(lane);
  u4 *out = reinterpret_cast<u4 *>(ws);
  // Products of keys with this wavefront's keys and queries, transposed: rows j, columns i = 16 w + m.
  by_wave(w, [&](auto wave) {
    constexpr int W = wave;
    f4v kk[W + 1] = {}, att[W + 1] = {};
#pragma unroll
    for (int a = 0; a < NS; ++a) {
      const bf8 ki = row16<KD>(keys, W, a, at);
#pragma unroll
      for (int jb = 0; jb <= W; ++jb) {
        const bf8 kj = row16<KD>(keys, jb, a, at);
        kk[jb] = mfma16(kj, ki, kk[jb]);
        att[jb] = mfma16(kj, qi[a], att[jb]);
      }
    }
    meet();
    const double si = sums[i];
#pragma unroll
    for (int jb = 0; jb <= W; ++jb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * jb + 4 * g + r;
        const float decay = (j <= i ? __builtin_amdgcn_exp2f(static_cast<float>(si - sums[j])) : 0.0f) * betas[j];
        att[jb][r] = j <= i && i < len ? att[jb][r] * decay * p.scale : 0.0f;
        low[j * kPitch + i] = j < i ? kk[jb][r] * decay : 0.0f;
      }
    store_rows<W>(att, out + kGdrTriBytes / 16, nullptr, lane);
  });
  __syncthreads();
  // Blocks on the diagonal, all in one wavefront: lane (block g, column m) by substitution.
  if (w == 0) {
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = k == m ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < 15; ++j) {
      const float *col = low + (16 * g + j) * kPitch + 16 * g;
#pragma unroll
      for (int k = (j + 1) / 4; k < 4; ++k) {
        const f4v l = *reinterpret_cast<const f4v *>(col + 4 * k);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (4 * k + r > j) x[4 * k + r] = fmaf(-l[r], x[j], x[4 * k + r]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<f4v *>(diag + lane * kDiagPitch + 4 * k) = f4v{x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]};
  }
  __syncthreads();
  // The other blocks, right to left: T_Wj = -(sum over k > j of T_Wk L_kj) T_jj, in float32 and transposed.
  by_wave(w, [&](auto wave) {
    constexpr int W = wave;
    f4v t[W + 1] = {};
#pragma unroll
    for (int r = 0; r < 4; ++r) t[W][r] = diag[(16 * W + 4 * g + r) * kDiagPitch + m];
#pragma unroll
    for (int j = W - 1; j >= 0; --j) {
      f4v acc = {};
#pragma unroll
      for (int k = j + 1; k <= W; ++k) {
        const f4v l = *reinterpret_cast<const f4v *>(low + (16 * j + m) * kPitch + 16 * k + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc = mfma_f32(l[r], t[k][r], acc);
      }
      const f4v d = *reinterpret_cast<const f4v *>(diag + (16 * j + m) * kDiagPitch + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) t[j] = mfma_f32(-d[r], acc[r], t[j]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (4 * g + r == m) t[W][r] = 0.0f;  // the ones stay out of what is rounded
    store_rows<W>(t, out, p.rest != nullptr ? reinterpret_cast<u4 *>(p.rest + id * kGdrRestBytes) : nullptr, lane);
  });
}

// ---------------------------------------------------------------------------
// From chunk to chunk
// ---------------------------------------------------------------------------

// A workgroup takes 32 columns (value elements) of a head from chunk to chunk.
// What a chunk has to wait for is the state, so two wavefronts do nothing but
// carry that, 16 columns each, and two others make y from the operands that
// those leave in LDS, and copy the next chunk there: each of the four has a
// SIMD to itself.  LAST: the last state is returned, and held to float32.  A
// chunk takes 2.4 us then (keys of 64: 1.8), 3.0 with a workgroup on every
// compute unit, 2100 cycles of which are the state's own matrix instructions,
// else 1.7 (1.5) with 1300; the rest is its operands' way through LDS and the
// splitting into parts.  With what the backward needs 3.2.
template <int KD, bool LAST>
__global__ void __launch_bounds__(256) gdr_fwd_kernel(const GdrParams p) {
  constexpr int NT = 64 * kPairs, NC = 16 * kPairs, NS = KD / 32, NB = KD / 16;
  constexpr unsigned kRows = 64 * KD * 2, kValues = 64 * NC * 2;
  constexpr unsigned kAtQ = kRows, kAtV = 2 * kRows, kAtW = kAtV + kValues, kBuffer = kAtW + kGdrChunkBytes;
  constexpr unsigned kState = NS * 2 * 1024, kUpdate = 2 * 2 * 1024;  // operands of the state and of z, of a wavefront
  __shared__ __align__(16) u4 lds[(2 * kBuffer + kPairs * (kState + kUpdate)) / 16];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave % kPairs;
  const unsigned vtiles = static_cast<unsigned>(p.vdim) / NC;
  const HeadTile which = head_tile(blockIdx.x, static_cast<unsigned>(p.batch * p.nheads), vtiles * static_cast<unsigned>(p.seg.count));
  const int64_t vt = which.tile % vtiles, bh = which.head, b = bh / p.nheads, h = bh % p.nheads;
  // Chunks first .. n - 1 of the row, of this segment.
  const int segment = static_cast<int>(which.tile / vtiles), len = gdr_length(p.lengths, b, p.seqlen);
  const int first = segment * static_cast<int>(p.seg.chunks), all = (len + 63) / 64;
  const int n = all < first + p.seg.chunks ? all : first + static_cast<int>(p.seg.chunks);
  const int col0 = static_cast<int>(vt) * NC + 16 * w;
  const unsigned base = lds_at(lds), parts_s = base + 2 * kBuffer + w * kState + lane * 16;
  const unsigned parts_z = base + 2 * kBuffer + kPairs * kState + w * kUpdate + lane * 16;
  const Lanes16 at = lanes16_of<KD>(lane);
  typedef __attribute__((address_space(3))) u4 lds16;

  if (wave < kPairs) {
    // The state: column col0 + m, key elements 32 a + 8g + 4x + r.
    f4v s[NB];
    const int64_t state = (bh * p.vdim + col0 + m) * KD + 8 * g;
    // (Not from h0 where there are segments: the last one's workgroup may write h_last in its place.)
    const float *from = p.seg.count > 1 ? p.ws_state + ((bh * p.seg.count + segment) * p.vdim + col0 + m) * KD + 8 * g
                        : p.h0 != nullptr ? p.h0 + state
                                          : nullptr;
    const bool begins = from != nullptr && (first < n || segment == 0);
#pragma unroll
    for (int j = 0; j < NB; ++j) s[j] = begins ? *reinterpret_cast<const f4v *>(from + 32 * (j / 2) + 4 * (j % 2)) : f4v{};
    // T's third part comes from memory to registers, a chunk ahead: there is no room for it in LDS.
    bf8 t3[kGdrFrags];
    if (LAST && first < n) load_rest(t3, p.rest + (bh * p.chunks + first) * kGdrRestBytes, lane);
    for (int c = first; c < n; ++c) {
      decltype(split<LAST>(s[0], s[0])) sp[NS];
#pragma unroll
      for (int a = 0; a < NS; ++a) {
        sp[a] = split<LAST>(s[2 * a], s[2 * a + 1]);
        *(lds16 *)(parts_s + a * 2048) = __builtin_bit_cast(u4, sp[a].hi);
        *(lds16 *)(parts_s + a * 2048 + 1024) = __builtin_bit_cast(u4, sp[a].lo);
      }
      meet();
      const unsigned tile = base + (c & 1) * kBuffer, tri_t = tile + kAtW, gates = tri_t + 2 * kGdrTriBytes + 16 * g;
      // Operands are read ahead of their use, in its order.
      bf8 ka[NS][4], kt[2][NB];
      decltype(split<LAST>(s[0], s[0])) tf[kGdrFrags];
      sh4 vf[4];
      f4v into[4];
#pragma unroll
      for (int a = 0; a < NS; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) ka[a][i] = row16<KD>(tile, i, a, at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vf[i] = rows4<NC>(tile + kAtV, i, w, lane);
        into[i] = lds_f4(gates + 256 + 64 * i);
      }
#pragma unroll
      for (int f = 0; f < kGdrFrags; ++f) {
        tf[f].hi = frag16(tri_t, f, lane);
        tf[f].lo = frag16(tri_t, kGdrFrags + f, lane);
        if constexpr (LAST) tf[f].rest = t3[f];
      }
      if (LAST && c + 1 < n) load_rest(t3, p.rest + (bh * p.chunks + c + 1) * kGdrRestBytes, lane);
      __builtin_amdgcn_sched_barrier(0);
      f4v x[4] = {};
#pragma unroll
      for (int a = 0; a < NS; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul_exact(ka[a][i], sp[a], x[i]);
      // v - e^G x, and z = T of that
      f4v z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int r = 0; r < 4; ++r) x[i][r] = fmaf(-into[i][r], x[i][r], up(vf[i][r]));
        z[i] = x[i];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const auto xp = split<LAST>(x[2 * k], x[2 * k + 1]);
#pragma unroll
        for (int i = 2 * k; i < 4; ++i) z[i] = mul_parts(tf[tri(i, k)], xp, z[i]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NB; ++j) kt[k][j] = col16<KD>(tile, j, k, at);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Parts zp = parts(z[2 * k], z[2 * k + 1]);
        *(lds16 *)(parts_z + k * 2048) = __builtin_bit_cast(u4, zp.hi);
        *(lds16 *)(parts_z + k * 2048 + 1024) = __builtin_bit_cast(u4, zp.lo);
      }
      meet();
      // s = e^GC s + sum over tokens of k (beta e^(GC - G) z)
      const float whole = lds_f4(tri_t + 2 * kGdrTriBytes + 256 + 240)[3];
#pragma unroll
      for (int j = 0; j < NB; ++j) s[j] *= whole;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f4v o0 = lds_f4(gates + 512 + 128 * k), o1 = lds_f4(gates + 512 + 128 * k + 64);
        const auto zp = split<LAST>(z[2 * k] * o0, z[2 * k + 1] * o1);
#pragma unroll
        for (int j = 0; j < NB; ++j) s[j] = mul_exact(kt[k][j], zp, s[j]);
      }
    }
    if (p.h_last != nullptr && ((n == all && first < n) || (all == 0 && segment == 0))) {
#pragma unroll
      for (int j = 0; j < NB; ++j) *reinterpret_cast<f4v *>(p.h_last + state + 32 * (j / 2) + 4 * (j % 2)) = s[j];
    }
    return;
  }

  const int id = tid - NT;
  const int64_t hk = h / (p.nheads / p.nqk), yt = p.nheads * p.vdim;
  const uint16_t *kp = p.k + b * p.k_batch + hk * KD, *qp = p.q + b * p.q_batch + hk * KD;
  const uint16_t *vp = p.v + b * p.v_batch + h * p.vdim + vt * NC;
  const char *ws = p.ops + bh * p.chunks * p.ops_step;
  uint16_t *yp = p.y + (b * p.seqlen * p.nheads + h) * p.vdim + col0;
  TileCopy<KD, NT> k_copy, q_copy;
  TileCopy<NC, NT> v_copy;
  k_copy.init(p.k_token, id);
  q_copy.init(p.q_token, id);
  v_copy.init(p.v_token, id);
  RowStore y_store;
  y_store.init(yt, lane);
  auto fetch_rows = [&](int c) {
    u4 *to = lds + (c & 1) * (kBuffer / 16);
    const int last = len - 1 - 64 * c;
    k_copy.start(to, kp + 64 * c * p.k_token, last, id);
    q_copy.start(to + kAtQ / 16, qp + 64 * c * p.q_token, last, id);
    v_copy.start(to + kAtV / 16, vp + 64 * c * p.v_token, last, id);
  };
  auto fetch_ws = [&](int c) {
    copy_share<kGdrChunkBytes / 1024, kPairs>(base + (c & 1) * kBuffer + kAtW, ws + c * p.ops_step, w, lane * 16);
  };
  if (first < n) {
    fetch_rows(first);
    fetch_ws(first);
  }
  f4v o[4];
  // What the backward starts from, whose operands have the values as k: each of
  // the two wavefronts turns half of both columns' tiles round.
  bf8 zt[2][2];
  const unsigned all_s = base + 2 * kBuffer, all_z = all_s + kPairs * kState;
  const int64_t nv = p.vdim / 32;
  auto saved = [&](int c) { return p.saved + (bh * p.chunks + c) * static_cast<int64_t>(gdr_saved_bytes(KD, p.vdim)) + lane * 16; };
  auto store = [&](int c) {
    const int64_t rest = p.seqlen - 64 * static_cast<int64_t>(c);
    y_store.put(yp + 64 * c * yt, rest < 64 ? static_cast<int>(rest) : 64, o);
    if (p.saved != nullptr) {
      // (Not through the caches, which the keys and operands are in: 118 -> 113 us at 4 x 2048 tokens, 16 heads of 128.)
      char *to = saved(c) + gdr_state_bytes(KD, p.vdim) + vt * 8192;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int part = 0; part < 2; ++part) __builtin_nontemporal_store(zt[i][part], reinterpret_cast<bf8 *>(to + (2 * i + w) * 2048 + part * 1024));
    }
  };
  for (int c = first; c < n; ++c) {
    // (Stores may be done before or after older copies, so the wait is for both.)
    arrive();
    if (c + 1 < n) fetch_rows(c + 1);
    const unsigned tile = base + (c & 1) * kBuffer, tri_a = tile + kAtW + kGdrTriBytes, gates = tri_a + kGdrTriBytes + 16 * g;
    bf8 qa[NS][4];
    Parts sp[NS], af[kGdrFrags];
    f4v qs[4];
#pragma unroll
    for (int a = 0; a < NS; ++a) {
      sp[a] = {__builtin_bit_cast(bf8, *(const lds16 *)(parts_s + a * 2048)),
               __builtin_bit_cast(bf8, *(const lds16 *)(parts_s + a * 2048 + 1024))};
#pragma unroll
      for (int i = 0; i < 4; ++i) qa[a][i] = row16<KD>(tile + kAtQ, i, a, at);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) qs[i] = lds_f4(gates + 64 * i);
#pragma unroll
    for (int f = 0; f < kGdrFrags; ++f) af[f] = {frag16(tri_a, f, lane), frag16(tri_a, kGdrFrags + f, lane)};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f4v{};
#pragma unroll
    for (int a = 0; a < NS; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = mul_exact(qa[a][i], sp[a], o[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= qs[i];
    bf8 before[NB / 2][2];
    if (p.saved != nullptr)
#pragma unroll
      for (int j = 0; j < NB / 2; ++j)
#pragma unroll
        for (int part = 0; part < 2; ++part) before[j][part] = turned<true>(all_s, all_s + kState, 2 * j + w, part, lane);
    meet();
    if (p.saved != nullptr) {
      char *to = saved(c) + vt * 2048;
#pragma unroll
      for (int j = 0; j < NB / 2; ++j)
#pragma unroll
        for (int part = 0; part < 2; ++part) __builtin_nontemporal_store(before[j][part], reinterpret_cast<bf8 *>(to + (2 * j + w) * nv * 2048 + part * 1024));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Parts zp = {__builtin_bit_cast(bf8, *(const lds16 *)(parts_z + k * 2048)),
                        __builtin_bit_cast(bf8, *(const lds16 *)(parts_z + k * 2048 + 1024))};
#pragma unroll
      for (int i = 2 * k; i < 4; ++i) o[i] = mul_parts(af[tri(i, k)], zp, o[i]);
    }
    if (c + 1 < n) fetch_ws(c + 1);
    if (p.saved != nullptr)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int part = 0; part < 2; ++part) zt[i][part] = turned<false>(all_z, all_z + kUpdate, 2 * i + w, part, lane);
    if (64 * c + 64 > len) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (64 * c + 16 * i + 4 * g + r >= len) o[i][r] = 0.0f;
    }
    store(c);
  }
  const int64_t last = segment + 1 < p.seg.count ? 64 * (first + p.seg.chunks) : p.seqlen;  // the segment's rows behind the length
  for (int64_t row = 64 * static_cast<int64_t>(n > first ? n : first) + g; row < last && row < p.seqlen; row += 4) st(yp, row * yt + m, 0.0f);
}

// E and P of a segment: 64 columns a workgroup, of E (the values' columns, from
// a state of 0) or P (the columns of the unit matrix, without values).  The
// backward takes P alone, transposed, of all segments but the first and last.
template <int KD, bool BWD>
__global__ void __launch_bounds__(256, 2) gdr_segment_kernel(const GdrParams p) {
  constexpr int NT = 256, NC = 64, NS = KD / 32, NB = KD / 16;
  constexpr unsigned kRows = 64 * KD * 2, kAtV = kRows, kAtW = kAtV + 64 * NC * 2, kAtG = kAtW + kGdrTriBytes, kBuffer = kAtG + kGdrGateBytes;
  __shared__ __align__(16) u4 lds[2 * kBuffer / 16];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned vtiles = BWD ? 0 : static_cast<unsigned>(p.vdim) / NC, tiles = vtiles + KD / NC;
  const HeadTile which = head_tile(blockIdx.x, static_cast<unsigned>(p.batch * p.nheads), tiles * static_cast<unsigned>(p.seg.count - (BWD ? 2 : 1)));
  const int64_t bh = which.head, b = bh / p.nheads, h = bh % p.nheads, hk = h / (p.nheads / p.nqk);
  const int segment = static_cast<int>(which.tile / tiles) + (BWD ? 1 : 0), len = gdr_length(p.lengths, b, p.seqlen);
  const int first = segment * static_cast<int>(p.seg.chunks), n = first + static_cast<int>(p.seg.chunks);
  if (64 * static_cast<int64_t>(n) >= len) return;  // the row has no segment behind this one: all its chunks are whole, too
  const unsigned tile = which.tile % tiles;
  const bool values = !BWD && tile < vtiles;
  const int col = static_cast<int>(values ? tile : tile - vtiles) * NC + 16 * w + m;
  const uint16_t *kp = p.k + b * p.k_batch + hk * KD, *vp = p.v + b * p.v_batch + h * p.vdim + tile * NC;
  const char *ws = p.ops + bh * p.chunks * p.ops_step;
  const unsigned base = lds_at(lds);
  const Lanes16 at = lanes16_of<KD>(lane);
  TileCopy<KD, NT> k_copy;
  TileCopy<NC, NT> v_copy;
  k_copy.init(p.k_token, tid);
  v_copy.init(p.v_token, tid);
  auto fetch = [&](int c) {
    u4 *to = lds + (c & 1) * (kBuffer / 16);
    const char *wc = ws + c * p.ops_step;
    k_copy.start(to, kp + 64 * c * p.k_token, 63, tid);
    if (values) v_copy.start(to + kAtV / 16, vp + 64 * c * p.v_token, 63, tid);
    copy_share<kGdrTriBytes / 1024, 4>(base + (c & 1) * kBuffer + kAtW, wc, w, lane * 16);
    if (w < static_cast<int>(kGdrGateBytes / 1024))
      copy_kib<1>(__builtin_amdgcn_readfirstlane(base + (c & 1) * kBuffer + kAtG + w * 1024), uniform(wc + 2 * kGdrTriBytes + w * 1024), lane * 16);
  };
  fetch(first);
  bf8 t3[kGdrFrags], next[kGdrFrags];  // T's third part, a chunk ahead
  if (!BWD) load_rest(next, p.rest + (bh * p.chunks + first) * kGdrRestBytes, lane);
  f4v s[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) s[j][r] = !values && 32 * (j / 2) + 8 * g + 4 * (j % 2) + r == col ? 1.0f : 0.0f;
  for (int c = first; c < n; ++c) {
    arrive();
    if (c + 1 < n) fetch(c + 1);
    if (!BWD) {
#pragma unroll
      for (int f = 0; f < kGdrFrags; ++f) t3[f] = next[f];
      if (c + 1 < n) load_rest(next, p.rest + (bh * p.chunks + c + 1) * kGdrRestBytes, lane);
    }
    const unsigned buffer = base + (c & 1) * kBuffer, tri_t = buffer + kAtW, gates = buffer + kAtG + 16 * g;
    f4v x[4] = {};
#pragma unroll
    for (int a = 0; a < NS; ++a) {
      const auto sp = split<!BWD>(s[2 * a], s[2 * a + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = mul_exact(row16<KD>(buffer, i, a, at), sp, x[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f4v into = lds_f4(gates + 256 + 64 * i);
      const sh4 v = rows4<NC>(buffer + kAtV, i, w, lane);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[i][r] = fmaf(-into[r], x[i][r], values ? up(v[r]) : 0.0f);
    }
    f4v z[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const auto xp = split<!BWD>(x[2 * k], x[2 * k + 1]);
#pragma unroll
      for (int i = 2 * k; i < 4; ++i) {
        decltype(split<!BWD>(s[0], s[0])) tf;
        tf.hi = frag16(tri_t, tri(i, k), lane);
        tf.lo = frag16(tri_t, kGdrFrags + tri(i, k), lane);
        if constexpr (!BWD) tf.rest = t3[tri(i, k)];
        z[i] = mul_parts(tf, xp, z[i]);
      }
    }
    const float whole = lds_f4(buffer + kAtG + 256 + 240)[3];
#pragma unroll
    for (int j = 0; j < NB; ++j) s[j] *= whole;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const auto zp = split<!BWD>(z[2 * k] * lds_f4(gates + 512 + 128 * k), z[2 * k + 1] * lds_f4(gates + 512 + 128 * k + 64));
#pragma unroll
      for (int j = 0; j < NB; ++j) s[j] = mul_exact(col16<KD>(buffer, j, k, at), zp, s[j]);
    }
  }
  const int64_t seg = bh * p.seg.count + segment;
  if (values) {
    float *to = p.ws_state + ((seg + 1) * p.vdim + col) * KD + 8 * g;  // where the join reads it and puts the state itself
#pragma unroll
    for (int j = 0; j < NB; ++j) *reinterpret_cast<f4v *>(to + 32 * (j / 2) + 4 * (j % 2)) = s[j];
  } else if (BWD) {
    // P^T as the join's operands, [16 key elements in][32 out][part], 1 KiB each: as it lies.
    char *to = reinterpret_cast<char *>(p.ws_carry + seg * 2 * KD * KD) + (4 * tile + w) * NS * 2048 + lane * 16;
#pragma unroll
    for (int a = 0; a < NS; ++a) {
      const Parts sp = parts(s[2 * a], s[2 * a + 1]);
      *reinterpret_cast<bf8 *>(to + a * 2048) = sp.hi;
      *reinterpret_cast<bf8 *>(to + a * 2048 + 1024) = sp.lo;
    }
  } else {
    // P as the join's operands, [16 key elements out][32 in][part], 1 KiB each,
    // turned round in LDS: the first two parts, then the third.
    typedef __attribute__((address_space(3))) u4 lds16;
    const unsigned left = base + (w & ~1) * NS * 2048;
    char *to = reinterpret_cast<char *>(p.ws_carry + seg * 3 * KD * KD) + (2 * (tile - vtiles) + w / 2) * (3 * 1024) + lane * 16;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      meet();
#pragma unroll
      for (int a = 0; a < NS; ++a) {
        const Parts3 sp = parts3(s[2 * a], s[2 * a + 1]);
        *(lds16 *)(base + (w * NS + a) * 2048 + lane * 16) = __builtin_bit_cast(u4, pass == 0 ? sp.hi : sp.rest);
        if (pass == 0) *(lds16 *)(base + (w * NS + a) * 2048 + 1024 + lane * 16) = __builtin_bit_cast(u4, sp.lo);
      }
      meet();
#pragma unroll
      for (int i = 0; i < NB / 2; ++i)
#pragma unroll
        for (int part = 0; part < 2 - pass; ++part)
          *reinterpret_cast<bf8 *>(to + (2 * i + w % 2) * NS * (3 * 1024) + (2 * pass + part) * 1024) =
              turned<true>(left, left + NS * 2048, 2 * i + w % 2, part, lane);
    }
  }
}

// The state before each segment, P S + E of the one before: 16 columns a
// workgroup, a quarter of the key elements a wavefront.  Each takes its part of
// P from memory, one segment ahead, and the columns' state from LDS, where all
// four leave theirs.  1.7 us a segment (keys of 64: 0.5), 1.2 with two parts;
// with 64 columns a workgroup and P in LDS 4.3.  Backwards the dS behind each segment, P^T dS + E
// of the one behind, from the last but one's, which is there.
template <int KD, bool BWD>
__global__ void __launch_bounds__(256) gdr_join_kernel(const GdrParams p) {
  constexpr int NS = KD / 32, NB = KD / 16, NJ = NB / 4, NP = BWD ? 2 : 3, kFrag = NP * 1024;
  typedef std::conditional_t<BWD, Parts, Parts3> Split;
  __shared__ __align__(16) u4 lds[2][NS * NP * 64];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const HeadTile which = head_tile(blockIdx.x, static_cast<unsigned>(p.batch * p.nheads), static_cast<unsigned>(p.vdim) / 16);
  const int64_t bh = which.head, b = bh / p.nheads;
  const int col = static_cast<int>(which.tile) * 16 + m, len = gdr_length(p.lengths, b, p.seqlen);
  const int span = static_cast<int>(p.seg.chunks) * 64, n = (len + span - 1) / span;  // segments of this row
  const int steps = n - (BWD ? 2 : 1);
  if (BWD && steps < 1) return;
  // This wavefront's blocks of 16 key elements in a column: P's rows lie as its
  // products leave them (16 j + 4g + r), P^T's are put in the order of the state
  // in the chains (32 (j / 2) + 8g + 4 (j % 2) + r), which its columns have.
  auto place = [&](int j) { return BWD ? 32 * ((NJ * w + j) / 2) + 8 * g + 4 * ((NJ * w + j) % 2) : 16 * (NJ * w + j) + 4 * g; };
  auto row = [&](int j) { return BWD ? 32 * ((NJ * w + j) / 2) + 8 * (m >> 2) + 4 * ((NJ * w + j) % 2) + (m & 3) : 16 * (NJ * w + j) + m; };
  auto slot_of = [&](int i) { return p.ws_state + ((bh * p.seg.count + i) * p.vdim + col) * KD; };
  const char *carry = reinterpret_cast<const char *>(p.ws_carry + bh * p.seg.count * NP * KD * KD) + g * 256;
  f4v s[NJ], next[NJ];
  Split pp[NJ][NS];
  auto segment = [&](int t) { return BWD ? n - 2 - t : t; };
  auto fetch = [&](int t) {
    const int i = segment(t);
    const float *to = slot_of(BWD ? i - 1 : i + 1);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      next[j] = *reinterpret_cast<const f4v *>(to + place(j));
#pragma unroll
      for (int a = 0; a < NS; ++a) {
        const char *from = carry + static_cast<int64_t>(i) * NP * 2 * KD * KD + ((row(j) >> 4) * NS + a) * kFrag + (row(j) & 15) * 16;
        pp[j][a].hi = *reinterpret_cast<const bf8 *>(from);
        pp[j][a].lo = *reinterpret_cast<const bf8 *>(from + 1024);
        if constexpr (!BWD) pp[j][a].rest = *reinterpret_cast<const bf8 *>(from + 2048);
      }
    }
  };
  if (steps > 0) fetch(0);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    if constexpr (BWD) {
      s[j] = *reinterpret_cast<const f4v *>(slot_of(n - 2) + place(j));
    } else {
      s[j] = p.h0 != nullptr ? *reinterpret_cast<const f4v *>(p.h0 + (bh * p.vdim + col) * KD + place(j)) : f4v{};
      *reinterpret_cast<f4v *>(slot_of(0) + place(j)) = s[j];
    }
  }
  for (int t = 0; t < steps; ++t) {
    char *mine = reinterpret_cast<char *>(lds[t & 1]);
    const Split own = split<!BWD>(s[0], s[NJ - 1]);
    auto put = [&](int part, bf8 v) {
      if constexpr (NJ == 2) *reinterpret_cast<bf8 *>(mine + w * kFrag + part * 1024 + lane * 16) = v;
      else *reinterpret_cast<u2 *>(mine + w / 2 * kFrag + part * 1024 + lane * 16 + w % 2 * 8) = half_of(v, 0);
    };
    put(0, own.hi);
    put(1, own.lo);
    if constexpr (!BWD) put(2, own.rest);
    __syncthreads();  // (What is read here is written again after the next one.)
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] = next[j];
#pragma unroll
    for (int a = 0; a < NS; ++a) {
      Split sp;
      sp.hi = *reinterpret_cast<const bf8 *>(mine + a * kFrag + lane * 16);
      sp.lo = *reinterpret_cast<const bf8 *>(mine + a * kFrag + 1024 + lane * 16);
      if constexpr (!BWD) sp.rest = *reinterpret_cast<const bf8 *>(mine + a * kFrag + 2048 + lane * 16);
#pragma unroll
      for (int j = 0; j < NJ; ++j) s[j] = mul_parts(pp[j][a], sp, s[j]);
    }
    if (t + 1 < steps) fetch(t + 1);
    float *to = slot_of(BWD ? segment(t) - 1 : segment(t) + 1);
#pragma unroll
    for (int j = 0; j < NJ; ++j) *reinterpret_cast<f4v *>(to + place(j)) = s[j];
  }
}

// ---------------------------------------------------------------------------
// One token
// ---------------------------------------------------------------------------

// Sum over the 8 (KD = 128: 128 = 8 lanes of 16) lanes that share a row.
__device__ __forceinline__ float sum8(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, true));   // lanes 1 apart
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, true));   // 2 apart
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));  // the other half of 8
  return v;
}

// Bound by memory: the state is read and written once, in float32 throughout,
// and y = scale (a S q + u (k.q)) needs no second pass over it.  8 lanes share a
// row of the state (a value element), 32 rows a workgroup.  (Two rows per lane
// were no faster: 42.1 and 42.1 us at 64 sequences and 32 heads of 128, 195 and
// 182 at 256.)  64 sequences, 32 heads of 128: 48 us a call, 5.6 TB/s; 4
// sequences, 16 heads: 4.0 us, of a call's 10.
template <int KD, typename G>
__global__ void __launch_bounds__(256) gdr_step_kernel(const GdrParams p) {
  constexpr int NP = KD / 32;  // pieces of 4 floats per lane
  const int tid = threadIdx.x, e = tid & 7;
  const unsigned vtiles = static_cast<unsigned>(p.vdim) / 32;
  const int64_t vt = blockIdx.x % vtiles, bh = blockIdx.x / vtiles, b = bh / p.nheads, h = bh % p.nheads;
  const int64_t hk = h / (p.nheads / p.nqk);
  const int row = static_cast<int>(vt) * 32 + (tid >> 3);
  f4v s[NP], k[NP], q[NP];
  const float *from = p.h0 + (bh * p.vdim + row) * KD + 4 * e;
#pragma unroll
  for (int a = 0; a < NP; ++a) s[a] = *reinterpret_cast<const f4v *>(from + 32 * a);
  float kq = 0.0f;
#pragma unroll
  for (int a = 0; a < NP; ++a) {
    const uint2 kb = *reinterpret_cast<const uint2 *>(p.k + b * p.k_batch + hk * KD + 32 * a + 4 * e);
    const uint2 qb = *reinterpret_cast<const uint2 *>(p.q + b * p.q_batch + hk * KD + 32 * a + 4 * e);
    k[a] = f4v{__uint_as_float(kb.x << 16), __uint_as_float(kb.x & 0xffff0000u), __uint_as_float(kb.y << 16),
               __uint_as_float(kb.y & 0xffff0000u)};
    q[a] = f4v{__uint_as_float(qb.x << 16), __uint_as_float(qb.x & 0xffff0000u), __uint_as_float(qb.y << 16),
               __uint_as_float(qb.y & 0xffff0000u)};
#pragma unroll
    for (int r = 0; r < 4; ++r) kq = fmaf(k[a][r], q[a][r], kq);
  }
  kq = sum8(kq);
  const float decay = __builtin_amdgcn_exp2f(gate<G>(p.g, bh) * kLog2e), beta = gate<G>(p.beta, bh);
  float *to = p.h_last + (bh * p.vdim + row) * KD + 4 * e;
  float sk = 0.0f, sq = 0.0f;
#pragma unroll
  for (int a = 0; a < NP; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sk = fmaf(s[a][i], k[a][i], sk);
      sq = fmaf(s[a][i], q[a][i], sq);
    }
  sk = sum8(sk);
  sq = sum8(sq);
  const float u = beta * fmaf(-decay, sk, ld(p.v, b * p.v_batch + h * p.vdim + row));
#pragma unroll
  for (int a = 0; a < NP; ++a) *reinterpret_cast<f4v *>(to + 32 * a) = s[a] * decay + k[a] * u;
  if (e == 0) st(p.y, bh * p.vdim + row, p.scale * fmaf(decay, sq, u * kq));
}

template <int KD, typename G>
void chunks(const GdrParams &p, hipStream_t s) {
  const dim3 n(static_cast<uint32_t>(p.batch * p.nheads * p.chunks));
  hipLaunchKernelGGL((gdr_chunk_kernel<KD, G>), n, dim3(256), 0, s, p);
}

template <int KD>
hipError_t fwd(const GdrParams &p, hipStream_t s) {
  const int64_t heads = p.batch * p.nheads;
  if (p.chunks > 0) p.gates_bf16 ? chunks<KD, uint16_t>(p, s) : chunks<KD, float>(p, s);
  if (p.seg.count > 1) {
    const int64_t parts = heads * (p.seg.count - 1) * ((p.vdim + KD) / 64);
    hipLaunchKernelGGL((gdr_segment_kernel<KD, false>), dim3(static_cast<uint32_t>(parts)), dim3(256), 0, s, p);
    hipLaunchKernelGGL((gdr_join_kernel<KD, false>), dim3(static_cast<uint32_t>(heads * (p.vdim / 16))), dim3(256), 0, s, p);
  }
  const dim3 n(static_cast<uint32_t>(heads * (p.vdim / 32) * p.seg.count));
  if (p.h_last != nullptr) hipLaunchKernelGGL((gdr_fwd_kernel<KD, true>), n, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((gdr_fwd_kernel<KD, false>), n, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int KD>
void bwd_carry(const GdrParams &p, hipStream_t s) {
  const int64_t parts = p.batch * p.nheads * (p.seg.count - 2) * (KD / 64);
  hipLaunchKernelGGL((gdr_segment_kernel<KD, true>), dim3(static_cast<uint32_t>(parts)), dim3(256), 0, s, p);
}

template <int KD>
void bwd_join(const GdrParams &p, hipStream_t s) {
  const int64_t groups = p.batch * p.nheads * (p.vdim / 16);
  hipLaunchKernelGGL((gdr_join_kernel<KD, true>), dim3(static_cast<uint32_t>(groups)), dim3(256), 0, s, p);
}

template <int KD, typename G>
hipError_t step(const GdrParams &p, hipStream_t s) {
  const int64_t heads = p.batch * p.nheads;
  hipLaunchKernelGGL((gdr_step_kernel<KD, G>), dim3(static_cast<uint32_t>(heads * (p.vdim / 32))), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

GdrSegments gdr_segments(int64_t heads, int64_t kdim, int64_t vdim, int64_t chunks) {
  // Times in us, between those with the last state and those without.  In turn a
  // chunk takes 2.4 or 1.7 (keys of 64: 1.8, 1.5).  With G segments each is gone
  // through twice, once for E and P (a compute unit has two workgroups of these,
  // and they are faster together) and once for y (it has one), and the join
  // takes a step per segment.  Calls with the last state, measured: 16 heads of
  // 128, 8192 tokens: 1 segment 336, 4 208, 8 195, 16 212; 2 heads of 64, 16384
  // tokens: 1 480, 32 73, 64 77; 32 heads of 128, 4096 tokens: 1 185, 2 205, 4
  // 186; without it 247, 186, 177, 193; 389, 69, 75; 141, 181, 165.
  const bool wide = kdim == 128;
  const int64_t columns = heads * (vdim / 32), pairs = heads * ((vdim + kdim) / 64);
  const double a = wide ? 2.6 : 1.65;
  auto rounds = [](int64_t n, int64_t room) { return static_cast<double>((n + room - 1) / room); };
  int64_t best = 1;
  double least = (wide ? 2.3 : 1.6) * static_cast<double>(chunks) + 4.0;
  for (int64_t g = 2; g <= 64 && g <= chunks && columns * g <= 512; ++g) {
    const double each = static_cast<double>((chunks + g - 1) / g);
    const int64_t n = pairs * (g - 1);
    const double first = n <= 256 ? a * each + 4.0 : (1.55 * a * each + 4.0) * rounds(n, 512);
    const double us = first + (a * each + 4.0) * rounds(columns * g, 256) + 4.0 + (wide ? 1.65 : 0.55) * static_cast<double>(g);
    if (us < least) {
      least = us;
      best = g;
    }
  }
  const int64_t each = (chunks + best - 1) / best;
  return {each > 0 ? (chunks + each - 1) / each : 1, each > 0 ? each : 1};
}

void launch_gdr_bwd_carry(const GdrParams &p, hipStream_t s) { p.kdim == 64 ? bwd_carry<64>(p, s) : bwd_carry<128>(p, s); }
void launch_gdr_bwd_join(const GdrParams &p, hipStream_t s) { p.kdim == 64 ? bwd_join<64>(p, s) : bwd_join<128>(p, s); }

GdrSizes gdr_sizes(const GdrParams &p) {
  const size_t heads = static_cast<size_t>(p.batch) * p.nheads, n = p.seg.count > 1 ? heads * p.seg.count : 0;
  return {heads * p.chunks * kGdrChunkBytes, heads * p.chunks * kGdrRestBytes, n * p.vdim * p.kdim * 4, n * 3 * p.kdim * p.kdim * 2};
}

hipError_t launch_gdr_fwd(const GdrParams &p, hipStream_t s) { return p.kdim == 64 ? fwd<64>(p, s) : fwd<128>(p, s); }

hipError_t launch_gdr_step(const GdrParams &p, hipStream_t s) {
  if (p.kdim == 64) return p.gates_bf16 ? step<64, uint16_t>(p, s) : step<64, float>(p, s);
  return p.gates_bf16 ? step<128, uint16_t>(p, s) : step<128, float>(p, s);
}

}  // namespace ssmb
