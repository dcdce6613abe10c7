// Backward of sliding-window attention with sinks for gfx950.
//
//   p_tj = exp(scale q_t.k_j - lse_t), dp_tj = dy_t.v_j
//   ds_tj = p_tj (dp_tj - dy_t.y_t)
//   dq_t = scale sum_j ds_tj k_j, dk_j = scale sum_t ds_tj q_t, dv_j = sum_t p_tj dy_t
//
// Two kernels, so that every sum has one owner and no atomics: one walks the
// keys of 32 queries per wavefront (dq), the other the queries and heads of 32
// keys per wavefront (dk, dv).  That is 7 products of pairs x headdim against
// the 5 that a single pass would need, which would have to add dq from many
// workgroups.  p and ds go from one product's result into the next one's
// operand as they lie (see swa_tile.h); both are rounded to bfloat16 there, as
// the matrix cores take them, and everything is summed in float32.
#include "swa_tile.h"

namespace ssmb {
namespace {

// dq; also log2(e) lse and dy.y of every query for the kernel below.
template <int D>
__global__ void __launch_bounds__(256, 2) swa_dq_kernel(const SwaParams p, int hw, unsigned qtiles, unsigned n) {
  constexpr int CH = D / 8, NB = D / 32, NS = D / 16;
  __shared__ __align__(16) u4 lds[2][2][kTile * CH];  // buffer, K or V
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned nheads = static_cast<unsigned>(p.nheads), nkv = static_cast<unsigned>(p.nkv);
  const unsigned group = nheads / nkv, hb = group / hw;
  const unsigned id = xcd_order(blockIdx.x, n);
  const unsigned qt = id % qtiles, rest = id / qtiles;
  const int64_t b = rest / (hb * nkv), c = rest / hb % nkv;
  const int64_t head = c * group + (rest % hb) * hw + wave % hw;
  const int qspan = 32 * (4 / hw), q0 = static_cast<int>(qt) * qspan, wq0 = q0 + 32 * (wave / hw);
  const int len = row_length(p, b), last = len - 1, t = wq0 + (lane & 31), L = static_cast<int>(p.seqlen);
  const int window = static_cast<int>(p.window), sinks = static_cast<int>(p.sinks);
  const int64_t out = ((b * p.seqlen + t) * p.nheads + head) * D;

  f16v dq[NB] = {};
  if (q0 < len) {
    const int qlast = q0 + qspan - 1 < last ? q0 + qspan - 1 : last;
    const KeyRow keys = key_row(q0, window, sinks);
    const int tiles = (keys.first + qlast - keys.low) / kTile + 1;
    const uint16_t *kp = p.k + b * p.k_batch + c * D, *vp = p.v + b * p.v_batch + c * D;
    auto start = [&](int i) {
      load_keys<D, 256>(lds[i & 1][0], kp, p.k_token, keys, i * kTile, last, tid);
      load_keys<D, 256>(lds[i & 1][1], vp, p.v_token, keys, i * kTile, last, tid);
    };
    bf8 q[NS], dy[NS];
    const int row = t < last ? t : last;
    const int64_t at = ((b * p.seqlen + row) * p.nheads + head) * D;
    const u4 *qs = reinterpret_cast<const u4 *>(p.q + b * p.q_batch + row * p.q_token + head * D);
    const u4 *ds = reinterpret_cast<const u4 *>(p.dy + at), *ys = reinterpret_cast<const u4 *>(p.y + at);
    float delta = 0.0f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      q[s] = __builtin_bit_cast(bf8, qs[2 * s + half]);
      dy[s] = __builtin_bit_cast(bf8, ds[2 * s + half]);
      const u4 d4 = ds[2 * s + half], y4 = ys[2 * s + half];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        delta = fmaf(__uint_as_float(d4[e] << 16), __uint_as_float(y4[e] << 16), delta);
        delta = fmaf(__uint_as_float(d4[e] & 0xffff0000u), __uint_as_float(y4[e] & 0xffff0000u), delta);
      }
    }
    delta += other_half(delta);
    const int64_t stat = (b * p.nheads + head) * p.seqlen + row;
    const float lse2 = p.lse[stat] * kLog2e, c2 = p.scale * kLog2e;
    if (half == 0 && t < len) {
      p.ws_lse2[stat] = lse2;
      p.ws_delta[stat] = delta;
    }
    const int own = sinks < t + 1 ? sinks : t + 1;
    start(0);
    for (int i = 0; i < tiles; ++i) {
      wait_tiles();
      __syncthreads();  // tile i has landed, and nobody reads the other buffer any more
      if (i + 1 < tiles) start(i + 1);
      const int v0 = i * kTile, j0 = keys.key(v0), j1 = keys.key(v0 + kTile - 1);
      const u4 *kt = lds[i & 1][0], *vt = lds[i & 1][1];
      if (j0 > wq0 + 31 || (j1 <= wq0 - window && j0 >= sinks) || wq0 >= len) continue;
      const bool whole = j1 <= wq0 && wq0 + 31 - j0 < window;
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        f16v s = {}, dp = {};
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) {
          s = mfma(row_operand<D>(kt, 32 * blk, ks, lane), q[ks], s);
          dp = mfma(row_operand<D>(vt, 32 * blk, ks, lane), dy[ks], dp);
        }
        reads_ahead<2 * NS>();
#pragma unroll
        for (int r = 0; r < 16; ++r)
          dp[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c2, -lse2)) * (dp[r] - delta);
        if (!whole) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int j = keys.key(v0 + 32 * blk + d_row(r, half));
            dp[r] = static_cast<unsigned>(t - j) < static_cast<unsigned>(window) || j < own ? dp[r] : 0.0f;
          }
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const bf8 dsk = as_operand(dp, ks);
#pragma unroll
          for (int db = 0; db < NB; ++db) dq[db] = mfma(col_operand<D>(kt, 32 * blk + 16 * ks, db, lane), dsk, dq[db]);
        }
      }
    }
  }
  if (t >= L) return;
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = static_cast<__bf16>(t < len ? dq[db][4 * j + r] * p.scale : 0.0f);
      *reinterpret_cast<bf4 *>(p.dq + out + 32 * db + 8 * j + 4 * half) = v;
    }
}

// dk and dv of 128 keys, 32 per wavefront, over a range of query tiles and
// heads (see SwaBwdPlan).
template <int D>
__global__ void __launch_bounds__(256, 2) swa_dkv_kernel(const SwaParams p, const SwaBwdPlan plan, unsigned n) {
  constexpr int CH = D / 8, NB = D / 32, NS = D / 16;
  __shared__ __align__(16) u4 lds[2][2][kTile * CH];  // buffer, Q or dy
  __shared__ __align__(16) float stats[2][2][kTile];  // buffer, log2(e) lse or dy.y
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned nkv = static_cast<unsigned>(p.nkv), group = static_cast<unsigned>(p.nheads) / nkv;
  const unsigned item = xcd_order(blockIdx.x, n);
  // Items of a (batch row, key head): sink blocks x chunks x slices, then the other blocks x slices.
  const unsigned per = plan.sink_blocks * plan.chunks * plan.slices + (plan.blocks - plan.sink_blocks) * plan.slices;
  const unsigned bc = item / per, k = item % per, slice = k % plan.slices, kb = k / plan.slices;
  const bool sink = kb < plan.sink_blocks * plan.chunks;
  const unsigned block = sink ? kb / plan.chunks : kb - plan.sink_blocks * plan.chunks + plan.sink_blocks;
  const unsigned chunk = sink ? kb % plan.chunks : 0;
  const int64_t b = bc / nkv, c = bc % nkv;
  const int heads = group / plan.slices, head0 = static_cast<int>(c * group + slice * heads);
  const int len = row_length(p, b), last = len - 1, L = static_cast<int>(p.seqlen);
  const int window = static_cast<int>(p.window), sinks = static_cast<int>(p.sinks);
  const int b0 = static_cast<int>(block) * 128, wk0 = b0 + 32 * wave, j = wk0 + (lane & 31);  // j: this lane's key
  const float c2 = p.scale * kLog2e;

  // Query tiles: from the block's own to the last that sees one of its keys.
  int t_lo = b0 / kTile, t_hi = 0;
  if (b0 < len) {
    const int reach = b0 < sinks || len - b0 <= window + 127 ? len : b0 + 127 + window;  // past the last query
    t_hi = (reach + kTile - 1) / kTile;
    if (sink) {
      t_lo += static_cast<int>(chunk * plan.chunk_tiles);
      const int end = t_lo + static_cast<int>(plan.chunk_tiles);
      t_hi = t_hi < end ? t_hi : end;
    }
  }
  const int nq = t_hi > t_lo ? t_hi - t_lo : 0, steps = nq * heads;

  f16v dk[NB] = {}, dv[NB] = {};
  if (steps > 0) {
    bf8 kf[NS], vf[NS];
    {
      const int row = j < last ? j : last;
      const u4 *ks = reinterpret_cast<const u4 *>(p.k + b * p.k_batch + row * p.k_token + c * D);
      const u4 *vs = reinterpret_cast<const u4 *>(p.v + b * p.v_batch + row * p.v_token + c * D);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        kf[s] = __builtin_bit_cast(bf8, ks[2 * s + half]);
        vf[s] = __builtin_bit_cast(bf8, vs[2 * s + half]);
      }
    }
    int at_head = head0, at_tile = t_lo;  // of the next tile to start
    auto start = [&](int i) {
      const int t0 = at_tile * kTile, buf = i & 1;
      load_tile<D, 256>(lds[buf][0], p.q + b * p.q_batch + at_head * D, p.q_token, t0, last, tid);
      load_tile<D, 256>(lds[buf][1], p.dy + (b * p.seqlen * p.nheads + at_head) * D, p.nheads * D, t0, last, tid);
      if (wave < 2) load_stats(stats[buf][wave], (wave == 0 ? p.ws_lse2 : p.ws_delta) + (b * p.nheads + at_head) * p.seqlen,
                               t0, last, lane);
      if (++at_tile == t_hi) {
        at_tile = t_lo;
        ++at_head;
      }
    };
    start(0);
    int tile = t_lo;
    for (int i = 0; i < steps; ++i) {
      wait_tiles();
      __syncthreads();
      if (i + 1 < steps) start(i + 1);
      const int t0 = tile * kTile;
      if (++tile == t_hi) tile = t_lo;
      const u4 *qt = lds[i & 1][0], *dt = lds[i & 1][1];
      const float *lse2 = stats[i & 1][0], *delta = stats[i & 1][1];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const int q0 = t0 + 32 * blk;
        // Does any of these 32 queries see any of the wavefront's keys, or all of them all?
        if (q0 + 31 < wk0 || (q0 >= wk0 + 31 + window && wk0 >= sinks) || q0 >= len || wk0 >= len) continue;
        const bool whole = q0 >= wk0 + 31 && q0 + 31 < len && (q0 + 31 - wk0 < window || wk0 + 31 < sinks);
        f16v s = {}, dp = {};
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) {
          s = mfma(row_operand<D>(qt, 32 * blk, ks, lane), kf[ks], s);
          dp = mfma(row_operand<D>(dt, 32 * blk, ks, lane), vf[ks], dp);
        }
        reads_ahead<2 * NS>();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 l4 = *reinterpret_cast<const float4 *>(lse2 + 32 * blk + 8 * g + 4 * half);
          const float4 d4 = *reinterpret_cast<const float4 *>(delta + 32 * blk + 8 * g + 4 * half);
          const float l[4] = {l4.x, l4.y, l4.z, l4.w}, d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            s[4 * g + r] = __builtin_amdgcn_exp2f(fmaf(s[4 * g + r], c2, -l[r]));
            dp[4 * g + r] = s[4 * g + r] * (dp[4 * g + r] - d[r]);
          }
        }
        if (!whole) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int t = q0 + d_row(r, half);
            const bool sees = t < len && (static_cast<unsigned>(t - j) < static_cast<unsigned>(window) || (j < sinks && j <= t));
            s[r] = sees ? s[r] : 0.0f;
            dp[r] = sees ? dp[r] : 0.0f;
          }
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const bf8 pk = as_operand(s, ks), dsk = as_operand(dp, ks);
#pragma unroll
          for (int db = 0; db < NB; ++db) {
            dv[db] = mfma(col_operand<D>(dt, 32 * blk + 16 * ks, db, lane), pk, dv[db]);
            dk[db] = mfma(col_operand<D>(qt, 32 * blk + 16 * ks, db, lane), dsk, dk[db]);
          }
        }
      }
    }
  }
  if (sink || plan.slices > 1) {
    // Terms of a sum over parts: [item][dk or dv][key][D] float32.
    float *part = p.ws_part + static_cast<int64_t>(item) * 2 * 128 * D + (32 * wave + (lane & 31)) * D;
#pragma unroll
    for (int db = 0; db < NB; ++db)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int e = 32 * db + 8 * g + 4 * half;
        *reinterpret_cast<float4 *>(part + e) =
            make_float4(dk[db][4 * g], dk[db][4 * g + 1], dk[db][4 * g + 2], dk[db][4 * g + 3]);
        *reinterpret_cast<float4 *>(part + 128 * D + e) =
            make_float4(dv[db][4 * g], dv[db][4 * g + 1], dv[db][4 * g + 2], dv[db][4 * g + 3]);
      }
    return;
  }
  if (j >= L) return;
  const int64_t out = ((b * p.seqlen + j) * p.nkv + c) * D;
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      bf4 a, v;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        a[r] = static_cast<__bf16>(j < len ? dk[db][4 * g + r] * p.scale : 0.0f);
        v[r] = static_cast<__bf16>(j < len ? dv[db][4 * g + r] : 0.0f);
      }
      *reinterpret_cast<bf4 *>(p.dk + out + 32 * db + 8 * g + 4 * half) = a;
      *reinterpret_cast<bf4 *>(p.dv + out + 32 * db + 8 * g + 4 * half) = v;
    }
}

// Sum the parts of the blocks that have them, in their order; one workgroup
// per (batch row, key head, block), a thread for 4 elements of a key.
template <int D>
__global__ void __launch_bounds__(256) swa_parts_kernel(const SwaParams p, const SwaBwdPlan plan, unsigned nsum) {
  const unsigned bc = blockIdx.x / nsum, block = blockIdx.x % nsum, nkv = static_cast<unsigned>(p.nkv);
  const unsigned per = plan.sink_blocks * plan.chunks * plan.slices + (plan.blocks - plan.sink_blocks) * plan.slices;
  const bool sink = block < plan.sink_blocks;
  const unsigned parts = plan.slices * (sink ? plan.chunks : 1);
  const int64_t first = static_cast<int64_t>(bc) * per +
                        (sink ? block * parts
                              : plan.sink_blocks * plan.chunks * plan.slices + (block - plan.sink_blocks) * plan.slices);
  const int64_t b = bc / nkv, c = bc % nkv;
  const int len = row_length(p, b), L = static_cast<int>(p.seqlen);
  for (int i = threadIdx.x; i < 128 * D / 4; i += 256) {
    const int j = static_cast<int>(block) * 128 + i / (D / 4);
    if (j >= L) break;
    float4 a = make_float4(0, 0, 0, 0), v = a;
    const float4 *part = reinterpret_cast<const float4 *>(p.ws_part + first * 2 * 128 * D) + i;
    for (unsigned k = 0; k < parts; ++k) {
      const float4 x = part[k * (128 * D / 2)], y = part[k * (128 * D / 2) + 128 * D / 4];
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
    }
    const float keep = j < len ? 1.0f : 0.0f, ka = keep * p.scale;
    const int64_t out = ((b * p.seqlen + j) * p.nkv + c) * D + i % (D / 4) * 4;
    const bf4 oa = {static_cast<__bf16>(a.x * ka), static_cast<__bf16>(a.y * ka), static_cast<__bf16>(a.z * ka),
                    static_cast<__bf16>(a.w * ka)};
    const bf4 ov = {static_cast<__bf16>(v.x * keep), static_cast<__bf16>(v.y * keep), static_cast<__bf16>(v.z * keep),
                    static_cast<__bf16>(v.w * keep)};
    *reinterpret_cast<bf4 *>(p.dk + out) = oa;
    *reinterpret_cast<bf4 *>(p.dv + out) = ov;
  }
}

template <int D>
hipError_t launch_d(const SwaParams &p, const SwaBwdPlan &plan, hipStream_t s) {
  const int64_t group = p.nheads / p.nkv;
  const int hw = group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1;
  const int64_t qspan = 32 * (4 / hw), qtiles = (p.seqlen + qspan - 1) / qspan;
  const int64_t n = qtiles * (group / hw) * p.nkv * p.batch, items = plan.items * p.batch * p.nkv;
  if (n > 0x7fffffff || items > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((swa_dq_kernel<D>), dim3(static_cast<uint32_t>(n)), dim3(256), 0, s, p, hw,
                     static_cast<unsigned>(qtiles), static_cast<unsigned>(n));
  hipLaunchKernelGGL((swa_dkv_kernel<D>), dim3(static_cast<uint32_t>(items)), dim3(256), 0, s, p, plan,
                     static_cast<unsigned>(items));
  const unsigned nsum = plan.slices > 1 ? plan.blocks : plan.sink_blocks;
  if (nsum > 0)
    hipLaunchKernelGGL((swa_parts_kernel<D>), dim3(static_cast<uint32_t>(nsum * p.batch * p.nkv)), dim3(256), 0, s, p, plan,
                       nsum);
  return hipGetLastError();
}

}  // namespace

SwaBwdPlan swa_bwd_plan(int64_t batch, int64_t seqlen, int64_t nheads, int64_t nkv, int64_t window, int64_t sinks) {
  SwaBwdPlan plan{};
  const int64_t blocks = (seqlen + 127) / 128;
  window = window < seqlen ? window : seqlen;
  sinks = sinks < seqlen ? sinks : seqlen;
  plan.blocks = static_cast<unsigned>(blocks);
  plan.chunks = 1;
  plan.slices = 1;
  const int64_t regular = (window + 127) / kTile + 1;  // query tiles that see a block through the window
  int64_t chunk = regular < 16 ? 16 : regular;
  const int64_t all = (seqlen + kTile - 1) / kTile;
  // Blocks that hold sinks are seen to the sequence's end: their queries are
  // cut into chunks of about an ordinary block's work.
  if (sinks > 0 && all > chunk) {
    plan.sink_blocks = static_cast<unsigned>((sinks + 127) / 128);
    plan.chunks = static_cast<unsigned>((all + chunk - 1) / chunk);
  }
  plan.chunk_tiles = static_cast<unsigned>(chunk);
  // Too few workgroups for the 256 CUs: the heads of a group are shared out.
  const int64_t group = nheads / nkv;
  int64_t slices = 1;
  while (slices < group && batch * nkv * blocks * slices < 512) {
    do ++slices;
    while (group % slices != 0);
  }
  plan.slices = static_cast<unsigned>(slices);
  plan.items = (static_cast<int64_t>(plan.sink_blocks) * plan.chunks + blocks - plan.sink_blocks) * slices;
  plan.has_parts = plan.sink_blocks > 0 || slices > 1;
  return plan;
}

hipError_t launch_swa_bwd(const SwaParams &p, const SwaBwdPlan &plan, hipStream_t s) {
  return p.headdim == 64 ? launch_d<64>(p, plan, s) : launch_d<128>(p, plan, s);
}

}  // namespace ssmb
