// Down to the rank: z = x A_l^T of the forward, u = dy B_l of the backward, for
// the rows of each adapter.
//
// A workgroup takes one piece of a run: up to 16 RF rows of one adapter, all r
// columns.  Its wavefronts split K, every NW-th chunk of 64 each, and their
// sums meet in LDS in their order.  What bounds it is reading x (or dy) once,
// as a stream of rows from anywhere: a row's 128 bytes of a chunk are whole
// lines.  A's rows (k contiguous) come straight into registers; B [N][r] is
// transposed on the way, through the wavefront's own LDS
// (ds_read_b64_tr_b16).  8192 tokens, 4096 wide, rank 16: 35 us forward, 28
// backward (2.2 and 2.7 TB/s; 28 and 24 where x and dy are in the cache); 7168
// wide, rank 64: 50 us, 171 MB from memory for 117 MB of x, since every piece
// reads its adapter's A again; 1001 tokens, 2880 wide, rank 32: 12 and 10 us, most of it the order's tables, the first rows and
// the sums, one after another.
#include "internal.h"
#include "proj.h"
#include "tile.h"

namespace moelora {

namespace {

constexpr int kChunk = 64;

struct ShrinkArgs {
  ProjArgs p;
  const uint16_t* in;  // [T][K]
  const uint16_t* w;   // KC: [L][r][K], else [L][K][r]
  uint16_t* parts;
  float* z;
  int K;
};

constexpr int shrink_threads(int nb) { return 64 * (nb <= 4 ? 8 : 4); }

// KC: the weights' k is contiguous.  NB: blocks of 16 columns.
template <bool KC, int NB, int RF>
struct Shrink {
  static constexpr int NT = shrink_threads(NB), NW = NT / 64;
  static constexpr int D = NB == 1 ? 4 : 2;           // chunks in flight
  static constexpr int WPL = 2 * NB;                  // 16-byte pieces of a chunk's weights per lane
  static constexpr int WBYTES = 64 * NB * 16 * 2 + 64;  // transposed: the wavefront's chunk, and what a read past r may see
  static constexpr int SUMS = RF * NB * 64 * 16;      // bytes of a wavefront's sums
  static constexpr int LDS = NW * (KC ? SUMS : std::max(SUMS, WBYTES));
};

template <bool KC, int NB, int RF>
__global__ __launch_bounds__(shrink_threads(NB)) void proj_shrink_kernel(ShrinkArgs a) {
  typedef Shrink<KC, NB, RF> C;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const ProjArgs& p = a.p;
  if ((int)blockIdx.x >= p.o.count[0]) return;
  const ProjItem item = p.o.shrink[blockIdx.x];
  const int lane = threadIdx.x & 63, l16 = lane & 15, kq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = p.r, K = a.K;

  // rows past the piece's and columns past r are zeros without traffic
  const buf_rsrc_t xs = make_rsrc(a.in, 0x7fffffffu), ws = make_rsrc(a.w, 0x7fffffffu);
  uint32_t xo[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    const int m = f * 16 + l16;
    xo[f] = m < item.n ? (uint32_t)p.o.perm[item.row + m] * (uint32_t)K * 2u + kq * 16u : kBufNone;
  }
  const uint32_t wbase = (uint32_t)item.adapter * (uint32_t)r * (uint32_t)K * 2u;
  uint32_t wo[C::WPL];
#pragma unroll
  for (int i = 0; i < C::WPL; ++i) {
    if (KC) {  // column block i / 2, 32-deep step i % 2
      const int j = (i >> 1) * 16 + l16;
      wo[i] = j < r ? wbase + (uint32_t)j * (uint32_t)K * 2u + (i & 1) * 64u + kq * 16u : kBufNone;
    } else {   // piece i of the chunk's 64 r values, which lie in a row
      wo[i] = (i * 64 + lane) * 8 < kChunk * r ? wbase + (i * 64u + lane) * 16u : kBufNone;
    }
  }

  struct Buf {
    u32x4_t x[RF][2], w[C::WPL];
  } q[C::D];
  const int chunks = (K + kChunk - 1) / kChunk;
  // Workgroups start at different chunks: rows lie a fixed distance apart, so
  // in step they would all ask the same memory channels.
  const int rot = (int)((blockIdx.x * (5u * C::NW)) % (unsigned)chunks);
  auto load = [&](int u, int i) __attribute__((always_inline)) {
    const int c = i + rot < chunks ? i + rot : i + rot - chunks;
    const int left = i < chunks ? K - c * kChunk : 0;  // of K; behind the last chunk nothing is fetched
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q[u].x[f][h] = ld16_buf(xs, h * 32 + kq * 8 < left && xo[f] != kBufNone ? xo[f] + (c * 2 + h) * 64u : kBufNone);
#pragma unroll
    for (int i = 0; i < C::WPL; ++i) {
      const bool in = KC ? (i & 1) * 32 + kq * 8 < left : (i * 64 + lane) * 8 < left * r;
      q[u].w[i] = ld16_buf(ws, in && wo[i] != kBufNone ? wo[i] + (uint32_t)c * (KC ? 128u : 128u * r) : kBufNone);
    }
    __builtin_amdgcn_sched_barrier(0);  // loads return in order: kept in the order of their use
  };
  f32x4_t acc[RF][NB];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[f][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  char* mine = smem + wave * C::WBYTES;
  auto mul = [&](int u) __attribute__((always_inline)) {
    if (!KC) {
#pragma unroll
      for (int i = 0; i < C::WPL; ++i)
        if ((i * 64 + lane) * 8 < kChunk * r) *reinterpret_cast<u32x4_t*>(mine + (i * 64 + lane) * 16) = q[u].w[i];
      asm volatile("" ::: "memory");  // a wavefront's LDS accesses run in order
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u32x4_t w;
        if (KC) {
          w = q[u].w[b * 2 + h];
        } else {
          // lane l takes k = 32 h + 8 (l / 16) + 0..7 of column 16 b + l % 16
          // (columns past r: another row's, dropped below)
          const char* at = mine + ((h * 32 + 8 * kq + ((lane >> 2) & 3)) * r + b * 16 + (lane & 3) * 4) * 2;
          const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
          const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * r * 2));
          const uint2 x = __builtin_bit_cast(uint2, lo), y = __builtin_bit_cast(uint2, hi);
          w = u32x4_t{x.x, x.y, y.x, y.y};
        }
#pragma unroll
        for (int f = 0; f < RF; ++f) acc[f][b] = mfma_16x16x32(q[u].x[f][h], w, acc[f][b]);
      }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int u = 0; u < C::D; ++u) load(u, wave + u * C::NW);
  for (int c = wave; c < chunks; c += C::D * C::NW) {
#pragma unroll
    for (int u = 0; u < C::D; ++u) {
      mul(u);
      load(u, c + (u + C::D) * C::NW);
    }
  }

  // the wavefronts' sums, added in their order; element i of a lane: row 4
  // (l / 16) + i, column l % 16
  __syncthreads();
  f32x4_t* part = reinterpret_cast<f32x4_t*>(smem);
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) part[(wave * RF * NB + f * NB + b) * 64 + lane] = acc[f][b];
  __syncthreads();
  const float s = proj_scale(p, item.adapter);
  for (int i = threadIdx.x; i < RF * NB * 64; i += C::NT) {
    f32x4_t v = part[i];
#pragma unroll
    for (int w = 1; w < C::NW; ++w) v += part[w * RF * NB * 64 + i];
    const int j = (i / 64 % NB) * 16 + (i & 15), m0 = (i / 64 / NB) * 16 + ((i & 63) >> 4) * 4;
    if (j >= r) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (m0 + e >= item.n) continue;
      const int64_t row = item.row + m0 + e;
      if (a.z) a.z[(int64_t)p.o.perm[row] * r + j] = v[e];
      uint16_t part[kParts];
      f32_to_bf16_three(s * v[e], part);
#pragma unroll
      for (int k = 0; k < kParts; ++k) a.parts[(row * kParts + k) * r + j] = part[k];
    }
  }
}

template <bool KC, int NB, int RF>
int launch_cfg(const ShrinkArgs& a, hipStream_t st) {
  typedef Shrink<KC, NB, RF> C;
  static std::atomic<uint64_t> attr_done;
  if (C::LDS > 65536) {
    const int rc = ensure_dynamic_lds(reinterpret_cast<const void*>(&proj_shrink_kernel<KC, NB, RF>), C::LDS, attr_done);
    if (rc) return rc;
  }
  const unsigned grid = (unsigned)proj_items(a.p.T, a.p.L, a.p.shrink_rows);
  proj_shrink_kernel<KC, NB, RF><<<grid, C::NT, C::LDS, st>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

template <bool KC>
int launch(const ShrinkArgs& a, hipStream_t st) {
  const int r = a.p.r;
  if (a.p.shrink_rows == 32) {
    if (r <= 16) return launch_cfg<KC, 1, 2>(a, st);
    if (r <= 32) return launch_cfg<KC, 2, 2>(a, st);
    return launch_cfg<KC, 4, 2>(a, st);
  }
  if (r <= 16) return launch_cfg<KC, 1, 1>(a, st);
  if (r <= 32) return launch_cfg<KC, 2, 1>(a, st);
  if (r <= 64) return launch_cfg<KC, 4, 1>(a, st);
  return launch_cfg<KC, 8, 1>(a, st);
}

}  // namespace

int launch_proj_shrink(const ProjArgs& p, bool back, const uint16_t* in, const uint16_t* weights, uint16_t* parts,
                       float* z, hipStream_t st) {
  const ShrinkArgs a{p, in, weights, parts, z, back ? p.N : p.K};
  return back ? launch<false>(a, st) : launch<true>(a, st);
}

}  // namespace moelora
