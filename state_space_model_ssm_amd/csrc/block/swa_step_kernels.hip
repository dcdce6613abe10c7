// One token of sliding-window attention against a ring cache, and the ring's
// fill from a prompt, for gfx950.
//
// The step reads the cache once, so it is bound by memory: a wavefront streams
// tiles of 64 slots into LDS of its own (no barriers between wavefronts; the
// next tile's keys start when this one's scores are done, its values when this
// one's products are), and the matrix cores take up to 32 heads of a group at
// once, padded, at a tenth of the time the bytes need.  So the weights, which a
// product takes in bfloat16, go through it in two parts, cut off and left over:
// y is then off by its own rounding alone (1.67e-3 of its norm, 2.1e-3 with
// rounded weights), for 1% of the time.  The slots of a (row, key head) are
// split over wavefronts and workgroups and joined by their maxima: in LDS
// within a workgroup, by a second launch across workgroups.
// 64 rows, 32 heads of 128 on 8, window 4096 (807 MB): 145 + 5 us, 5.6 TB/s.
#include "swa_step.h"

namespace ssmb {
namespace {

// Zeros in the rows from r on: they repeat the last slot, whose infinity, if it
// has one, would come out as 0 times itself.
template <int D>
__device__ __forceinline__ void clear_rows(u4 *tile, int r, int lane) {
  constexpr int CH = D / 8;
  for (int k = r + lane / CH; k < kTile; k += 64 / CH) tile[slot<D>(k, lane % CH)] = u4{};
}

// Weights (registers 8 s .. 8 s + 7 of a D result) as two operands whose sum
// they are to 2^-16: cut off after 8 bits, and what that leaves, which is held
// above 0, so that both times an infinity have its sign.
__device__ __forceinline__ void two_parts(const f16v &d, int s, bf8 &cut, bf8 &rest) {
  u4 c;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = d[8 * s + 2 * k], b = d[8 * s + 2 * k + 1];
    const unsigned ca = __float_as_uint(a) & 0xffff0000u, cb = __float_as_uint(b) & 0xffff0000u;
    c[k] = ca >> 16 | cb;
    rest[2 * k] = static_cast<__bf16>(fmaxf(a - __uint_as_float(ca), 0x1p-100f));
    rest[2 * k + 1] = static_cast<__bf16>(fmaxf(b - __uint_as_float(cb), 0x1p-100f));
  }
  cut = __builtin_bit_cast(bf8, c);
}

template <int D>
__global__ void __launch_bounds__(256) swa_step_kernel(const SwaStepParams p, unsigned splits, unsigned qblocks) {
  constexpr int CH = D / 8, NB = D / 32, NS = D / 16;
  constexpr int kCopies = kTile * CH / 64;  // copies of 1 KiB per tile
  __shared__ __align__(16) u4 lds[4][2][kTile * CH];  // wavefront, K or V; in the end o, [32][D] float32
  __shared__ float tops[4][32], sums[4][32];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned nkv = static_cast<unsigned>(p.nkv), group = static_cast<unsigned>(p.nheads) / nkv;
  const unsigned split = blockIdx.x % splits, rest = blockIdx.x / splits, qb = rest % qblocks, bc = rest / qblocks;
  const int64_t b = bc / nkv, c = bc % nkv;
  const int g0 = qb * 32, heads = static_cast<int>(group) - g0 < 32 ? static_cast<int>(group) - g0 : 32;
  const int slots = static_cast<int>(p.sinks + p.window), sinks = static_cast<int>(p.sinks);
  const int pos = p.pos[b];
  f16v o[NB] = {};
  float top = -INFINITY, sum = 0.0f;
  if (pos >= 0) {
    const int own = pos < sinks ? pos : sinks + (pos - sinks) % static_cast<int>(p.window);
    const int count = pos < slots ? pos + 1 : slots, last = count - 1;
    const int tiles = (count + kTile - 1) / kTile;
    // Tiles of this wavefront: an even share of the row's.
    const unsigned parts = splits * 4, part = split * 4 + wave;
    const unsigned each = tiles / parts, more = tiles % parts;
    const int lo = static_cast<int>(each * part + (part < more ? part : more));
    const int hi = lo + static_cast<int>(each + (part < more ? 1 : 0));
    const int64_t base = static_cast<int64_t>(bc) * slots * D;
    const uint16_t *kn = p.k + b * p.k_batch + c * D, *vn = p.v + b * p.v_batch + c * D;
    u4 *kt = lds[wave][0], *vt = lds[wave][1];
    const Lanes at = lanes_of<D>(lane);
    if (lo < hi) {
      bf8 q[NS];
      const int row = (lane & 31) < heads ? lane & 31 : 0;  // lanes past the group repeat its first head
      const u4 *src = reinterpret_cast<const u4 *>(p.q + b * p.q_batch + (c * group + g0 + row) * D);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        u4 v = src[2 * s + half];
        if (p.scale < 0.0f) v ^= 0x80008000u;  // a negative scale is taken as -q
        q[s] = __builtin_bit_cast(bf8, v);
      }
      const float c2 = fmaxf(fabsf(p.scale) * kLog2e, 0x1p-100f);
      load_tile<D, 64>(kt, p.k_cache + base, D, lo * kTile, last, lane);
      load_tile<D, 64>(vt, p.v_cache + base, D, lo * kTile, last, lane);
      for (int i = lo; i < hi; ++i) {
        const int k0 = i * kTile, mine = own - k0;  // the token's row in this tile, if within it
        const bool has = mine >= 0 && mine < kTile;
        wait_tiles<kCopies>();  // the keys: all but the copies of the values
        if (has) put_row<D>(kt, kn, mine, lane);
        f16v s[2] = {};
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int ks = 0; ks < NS; ++ks) s[blk] = mfma(row_operand<D>(kt, 32 * blk, ks, at), q[ks], s[blk]);
        wait_reads();
        if (i + 1 < hi) load_tile<D, 64>(kt, p.k_cache + base, D, k0 + kTile, last, lane);
        if (k0 + kTile > count) {
#pragma unroll
          for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (k0 + 32 * blk + d_row(r, half) >= count) s[blk][r] = -INFINITY;
        }
        to_weights(s, c2, o, top, sum);
        if (i + 1 < hi) wait_tiles<kCopies>();  // the values: all but the copies of the next keys
        else wait_tiles<0>();
        if (has) put_row<D>(vt, vn, mine, lane);
        if (k0 + kTile > count) clear_rows<D>(vt, count - k0, lane);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          bf8 cut, rest;
          two_parts(s[ks / 2], ks % 2, cut, rest);
#pragma unroll
          for (int db = 0; db < NB; ++db) {
            const bf8 v = col_operand<D>(vt, 16 * ks, db, at);
            o[db] = mfma(v, cut, o[db]);
            o[db] = mfma(v, rest, o[db]);
          }
        }
        wait_reads();
        if (i + 1 < hi) load_tile<D, 64>(vt, p.v_cache + base, D, k0 + kTile, last, lane);
        if (has && lane < CH) {  // the token takes its slot
          const int64_t to = base + static_cast<int64_t>(own) * D;  // own * D passes 2^31 in a long cache
          reinterpret_cast<u4 *>(p.k_cache + to)[lane] = reinterpret_cast<const u4 *>(kn)[lane];
          reinterpret_cast<u4 *>(p.v_cache + to)[lane] = reinterpret_cast<const u4 *>(vn)[lane];
        }
      }
    }
    sum += other_half(sum);
  }
  // Join the four wavefronts.
  float *mine = reinterpret_cast<float *>(lds[wave]);
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<float4 *>(mine + (lane & 31) * D + 32 * db + 8 * g + 4 * half) =
          make_float4(o[db][4 * g], o[db][4 * g + 1], o[db][4 * g + 2], o[db][4 * g + 3]);
  if (half == 0) {
    tops[wave][lane] = top;
    sums[wave][lane] = sum;
  }
  __syncthreads();
  for (int i = tid; i < heads * D; i += 256) {
    const int row = i / D, e = i % D;
    float best = tops[0][row];
#pragma unroll
    for (int w = 1; w < 4; ++w) best = fmaxf(best, tops[w][row]);
    // (A share without a maximum holds zeros, or the NaN that all its scores were.)
    float acc = 0.0f, all = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = tops[w][row] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(tops[w][row] - best);
      acc = fmaf(f, reinterpret_cast<const float *>(lds[w])[row * D + e], acc);
      all = fmaf(f, sums[w][row], all);
    }
    const int64_t head = b * p.nheads + c * group + g0 + row;
    if (splits == 1) {
      st(p.y, head * D + e, all == 0.0f ? 0.0f : acc / all);
    } else {
      p.ws_o[(head * splits + split) * D + e] = acc;
      if (e == 0) {
        p.ws_stat[(head * splits + split) * 2] = best;
        p.ws_stat[(head * splits + split) * 2 + 1] = all;
      }
    }
  }
}

// A thread takes 16 bytes of a slot at a time: slot s of a row of length n
// holds position s below the sinks, else the largest position p < n with
// (p - sinks) mod window = s - sinks.
__global__ void __launch_bounds__(256) swa_fill_kernel(const SwaParams p, uint16_t *kc, uint16_t *vc) {
  const int64_t chunks = p.headdim / 8, slots = p.sinks + p.window, all = p.batch * p.nkv * slots * chunks;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; id < all; id += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t e = id % chunks, s = id / chunks % slots, c = id / chunks / slots % p.nkv;
    const int64_t b = id / chunks / slots / p.nkv;
    int64_t n = p.lengths != nullptr ? p.lengths[b] : p.seqlen;
    n = n < 0 ? 0 : n > p.seqlen ? p.seqlen : n;
    int64_t pos = s;
    if (s >= n) continue;
    if (s >= p.sinks) pos += (n - 1 - s) / p.window * p.window;
    const uint4 k = *reinterpret_cast<const uint4 *>(p.k + b * p.k_batch + pos * p.k_token + c * p.headdim + e * 8);
    const uint4 v = *reinterpret_cast<const uint4 *>(p.v + b * p.v_batch + pos * p.v_token + c * p.headdim + e * 8);
    reinterpret_cast<uint4 *>(kc)[id] = k;
    reinterpret_cast<uint4 *>(vc)[id] = v;
  }
}

// Join the splits of a head, a thread per element.
template <int D>
__global__ void __launch_bounds__(D) swa_join_kernel(const SwaStepParams p, int splits) {
  const int64_t head = blockIdx.x;
  const float *stat = p.ws_stat + head * splits * 2, *part = p.ws_o + head * splits * D + threadIdx.x;
  float best = -INFINITY, acc = 0.0f, all = 0.0f;
  for (int k = 0; k < splits; ++k) best = fmaxf(best, stat[2 * k]);
  for (int k = 0; k < splits; ++k) {
    const float f = stat[2 * k] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(stat[2 * k] - best);
    acc = fmaf(f, part[k * D], acc);
    all = fmaf(f, stat[2 * k + 1], all);
  }
  st(p.y, head * D + threadIdx.x, all == 0.0f ? 0.0f : acc / all);
}

}  // namespace

int swa_step_splits(int64_t batch, int64_t nheads, int64_t nkv, int64_t slots) {
  // Four workgroups per CU even out rows of unequal length; a wavefront has at
  // least one tile.
  const int64_t rows = batch * nkv * ((nheads / nkv + 31) / 32), tiles = (slots + kTile - 1) / kTile;
  const int64_t want = (1024 + rows - 1) / (rows > 0 ? rows : 1), most = (tiles + 3) / 4;
  return static_cast<int>(want < most ? want : most);
}

hipError_t launch_swa_step(const SwaStepParams &p, int splits, hipStream_t s) {
  const unsigned qblocks = static_cast<unsigned>((p.nheads / p.nkv + 31) / 32);
  const dim3 g(static_cast<uint32_t>(p.batch * p.nkv * qblocks * splits)), t(256), gj(static_cast<uint32_t>(p.batch * p.nheads));
  const unsigned sp = static_cast<unsigned>(splits);
  if (p.headdim == 64) {
    hipLaunchKernelGGL((swa_step_kernel<64>), g, t, 0, s, p, sp, qblocks);
    if (splits > 1) hipLaunchKernelGGL((swa_join_kernel<64>), gj, dim3(64), 0, s, p, splits);
  } else {
    hipLaunchKernelGGL((swa_step_kernel<128>), g, t, 0, s, p, sp, qblocks);
    if (splits > 1) hipLaunchKernelGGL((swa_join_kernel<128>), gj, dim3(128), 0, s, p, splits);
  }
  return hipGetLastError();
}

hipError_t launch_swa_fill(const SwaParams &p, uint16_t *kc, uint16_t *vc, hipStream_t s) {
  const int64_t n = p.batch * p.nkv * (p.sinks + p.window) * (p.headdim / 8);
  if (n == 0) return hipSuccess;
  const int64_t groups = (n + 255) / 256 < kMaxGroups ? (n + 255) / 256 : kMaxGroups;
  hipLaunchKernelGGL(swa_fill_kernel, dim3(static_cast<uint32_t>(groups)), dim3(256), 0, s, p, kc, vc);
  return hipGetLastError();
}

}  // namespace ssmb
