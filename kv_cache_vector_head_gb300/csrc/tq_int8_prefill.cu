// Prefill attention over the pages of the 8-bit arm on the fifth-generation tensor cores (d = 128).
//
//   S = Q K^T, P = exp2(S f - m), O += P V over key tiles of 128 tokens; f = scale log2(e) ks of the token's page.
//
// A block owns up to 256 rows (query, head of the group) of one (sequence, KV head), so that a page is
// read from memory once for all of them.  Operands are f16: codes are exact, a query is exact (bf16, f16; scaled
// by a power of two a row) or two limbs (float), and the weights P vs are two limbs, since one f16 limb would
// leave 2^-12 of the float output: a tile costs one product for S (two for float queries) and two for O.
//
//   warps 0-3, 4-7   a unit each: one thread a row takes its S row from tensor memory (tcgen05.ld), keeps the
//                    running maximum and sum, and writes P's limbs over S; then adds the tile's O to its 128
//                    registers.  O starts anew in every tile: the tensor cores' accumulation truncates, which over a
//                    long context would cost 2^-25 of the output a step, float additions round.
//   warps 8-11       turn the tile's codes (and the float16 window rows) into f16 operands in shared memory, two
//                    tiles ahead.
//   warp 12          one thread issues tcgen05.mma; S_u of the next tile runs while the other unit is in its softmax.
// With one row tile (RT = 1: up to 128 rows, or float queries, whose second limb takes the second tile's
// shared memory) the units take the key tiles in turn and join at the end.
#include <math.h>

#include <algorithm>

#include "tq_int8.cuh"
#include "tq_launch.h"

namespace tq {

static __device__ unsigned int g_int8_prefill_err = 0;

namespace {

constexpr int D = 128;
constexpr int KT = 128;              // tokens of a key tile
constexpr int GROUPS = KT / kPage;
constexpr int kThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kWeightTop = 16384.f;

// Shared-memory operands without swizzle: core matrices of 8 rows x 16 bytes; LBO steps along the contraction
// (8 elements), SBO along the rows (8).
constexpr uint32_t kQLbo = 128, kQSbo = 2048, kQTile = 128 * D * 2;
constexpr uint32_t kKLbo = 144, kKSbo = 16 * 144;               // keys: rows tokens
constexpr uint32_t kVSbo = 144, kVLbo = 16 * 144 + 64;          // values: rows channels, contraction tokens
constexpr uint32_t kKTile = 16 * kKSbo, kVTile = 16 * kVLbo;
constexpr int kStages = 2;
constexpr uint32_t kSmemQ = 0, kSmemK = 2 * kQTile, kSmemV = kSmemK + kStages * kKTile;
constexpr uint32_t kSmemBytes = kSmemV + kStages * kVTile;
constexpr int kIdesc = (1 << 4) | ((128 >> 3) << 17) | ((128 >> 4) << 24);  // f16 x f16 -> f32, M = N = 128

struct Shared {
  uint64_t kfull[kStages], vfull[kStages], kfree[kStages], vfree[kStages];
  uint64_t sfull[2], pready[2], ofull[2], drained;
  float2 scale[kStages][GROUPS];  // key and value scale of a group of 16 tokens
  uint32_t live[kStages];         // groups whose page is there
  uint32_t bad[kStages][GROUPS];  // window tokens with non-finite values
  float rowscale[256];            // 1 / the power of two of a query row
  float m[128], l[128];
  uint32_t tmem;
  int fail;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
// Bounded wait (about a second): false when it ran out.
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity) {
  uint32_t done = 0;
  for (unsigned it = 0; it < (1u << 20) && !done; ++it)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(b)), "r"(parity), "n"(1000)
        : "memory");
  return done != 0;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | ((uint64_t)1 << 46);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(kIdesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(kIdesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(a));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(a));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(a)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float pow2_above(float s) { return __uint_as_float((__float_as_uint(s) + 0x007fffffu) & 0x7f800000u); }
__device__ __forceinline__ float pow2_inv(float v) { return __uint_as_float(0x7f000000u - __float_as_uint(v)); }

// RT row tiles of 128, QL query limbs (RT + QL = 3).  grid (row tiles, hkv, batch * splits).
template <int RT, int QL>
__global__ void __launch_bounds__(kThreads, 1)
    i8_prefill_attn_kernel(const __grid_constant__ KParams P, const __grid_constant__ KCache C, int n_query, const void* q,
                           int dtype, float scale, float* out, float* lse, unsigned char* ws, WsLayout L, int max_ctx) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y, S = L.n_comp_splits, b = blockIdx.z / S, split = blockIdx.z % S;
  const int G = P.G, rows = n_query * G;
  const int row0 = blockIdx.x * 128 * RT;
  const uint32_t sbase = smem_u32(smem);

  int n = C.seq_len[b], nc = C.n_compressed[b];
  {
    bool wrong = n < n_query || n > max_ctx || nc < 0 || nc > n || nc % kPage;
    n = min(max(n, 0), max_ctx);
    nc = min(max(nc, 0), n) / kPage * kPage;
    if (nc / kPage > C.max_pages || n - nc >= C.ring) {
      wrong = true;
      nc = min(nc, C.max_pages * kPage);
      n = min(n, nc + C.ring - 1);
    }
    if (wrong && tid == 0) atomicOr(&g_int8_prefill_err, TQ_DEVERR_SEQ_LEN);
  }
  const int seq = C.seq_len[b];
  // position of row r's query; the last row of the block sees the most
  auto row_pos = [&](int r) { return min((long long)seq - n_query + r / G, (long long)n - 1); };
  const int last = min(rows, row0 + 128 * RT) - 1;
  const int end = (int)max(0LL, row_pos(last) + 1);  // tokens that any row sees
  const int tiles = (end + KT - 1) / KT, per = (tiles + S - 1) / S;
  const int j0 = min(tiles, split * per), j1 = min(tiles, j0 + per);

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.kfull[i], 4);
      mbar_init(&sh.vfull[i], 4);
      mbar_init(&sh.kfree[i], 1);
      mbar_init(&sh.vfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pready[i], 128);
      mbar_init(&sh.ofull[i], 1);
    }
    mbar_init(&sh.drained, 1);
    sh.fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // ---- queries: a warp a row; the sign of the scale goes into them, so that larger stays larger
  const float sgn = scale < 0.f ? -1.f : 1.f;
  for (int r = warp; r < 128 * RT; r += kThreads / 32) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    const int rr = row0 + r;
    if (rr < rows && 4 * lane < P.dh) {
      const long long at = (((long long)b * n_query + rr / G) * P.hq + (long long)g * G + rr % G) * P.dh + 4 * lane;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = load_elem(q, dtype, at + e) * sgn;
    }
    const float a = warp_max_f(fmaxf(fmaxf(i8_mag(x[0]), i8_mag(x[1])), fmaxf(i8_mag(x[2]), i8_mag(x[3]))));
    const int e2 = a > 0.f ? min(max(140 - (int)(__float_as_uint(a) >> 23), -113), 126) : 0;
    const float up = __uint_as_float((uint32_t)(127 + e2) << 23);
    if (lane == 0) sh.rowscale[r] = __uint_as_float((uint32_t)(127 - e2) << 23);
    const uint32_t at = (uint32_t)(r >> 7) * kQTile + (uint32_t)((r & 127) >> 3) * kQSbo + (r & 7) * 16 + (lane >> 1) * kQLbo + (lane & 1) * 8;
    const __half2 h0 = __floats2half2_rn(x[0] * up, x[1] * up), h1 = __floats2half2_rn(x[2] * up, x[3] * up);
    *reinterpret_cast<uint2*>(smem + kSmemQ + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    if (QL == 2) {
      const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
      *reinterpret_cast<uint2*>(smem + kSmemQ + kQTile + at) =
          make_uint2(pack_f16(x[0] * up - f0.x, x[1] * up - f0.y), pack_f16(x[2] * up - f1.x, x[3] * up - f1.y));
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem;  // units' S / P at 0 and 128, their O at 256 and 384

  if (warp < 8) {
    // ------------------------------------------------------------ softmax of unit u
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int u = warp >> 2, r = tid & 127;
    const int rr = row0 + (RT == 2 ? u * 128 : 0) + r;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + 128u * u, to = tmem + lanes + 256u + 128u * u;
    const int pos = rr < rows ? (int)max(-1LL, row_pos(rr)) : -1;
    const float fq = sh.rowscale[(RT == 2 ? u * 128 : 0) + r] * fabsf(scale) * kLog2e;
    float o[D];
#pragma unroll
    for (int i = 0; i < D; ++i) o[i] = 0.f;
    float m = -INFINITY, l = 0.f, vref = 0.f;
    uint32_t ph = 0;
    bool failed = false;
    for (int j = j0 + (RT == 1 ? u : 0); j < j1; j += RT == 1 ? 2 : 1, ph ^= 1) {
      const int st = (j - j0) & 1, sp = ((j - j0) >> 1) & 1;
      if (!mbar_wait(&sh.vfull[st], sp) || !mbar_wait(&sh.sfull[u], ph)) {
        failed = true;
        break;
      }
      tc_after();
      const uint32_t live = sh.live[st];
      const int see = pos - j * KT;  // columns 0 .. see are visible
      float mx = -INFINITY, vn = vref;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        tmem_ld32(ts + 32 * c, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int gi = 2 * c + h;
          float a = -INFINITY;
          if (see >= 16 * gi + 15) {
#pragma unroll
            for (int i = 0; i < 16; ++i) a = fmaxf(a, __uint_as_float(v[16 * h + i]));
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (16 * gi + i <= see) a = fmaxf(a, __uint_as_float(v[16 * h + i]));
          }
          const float2 sc = sh.scale[st][gi];
          if (live >> gi & 1) mx = fmaxf(mx, a == -INFINITY ? a : a * (sc.x * fq));
          vn = fmaxf(vn, pow2_above(sc.y));
        }
      }
      const float mn = fmaxf(m, mx), mb = mn == -INFINITY ? 0.f : mn;
      const float al = ex2(m - mb);
      const float av = vn > 0.f ? al * (vref * pow2_inv(vn)) : al;
      const float vi = vn > 0.f ? pow2_inv(vn) : 0.f;
      m = mn;
      vref = vn;
      l *= al;
#pragma unroll
      for (int gi = 0; gi < GROUPS; ++gi) {
        uint32_t v[16], pk[16];
        tmem_ld16(ts + 16 * gi, v);
        const float2 sc = sh.scale[st][gi];
        const float f = sc.x * fq, wv = sc.y * vi * kWeightTop;
        const int lim = (live >> gi & 1) ? see - 16 * gi : -1;  // tokens 0 .. lim of the group
        float ls = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float e0 = ex2(fmaf(__uint_as_float(v[2 * i]), f, -mb)), e1 = ex2(fmaf(__uint_as_float(v[2 * i + 1]), f, -mb));
          if (lim < 15) {
            e0 = 2 * i <= lim ? e0 : 0.f;
            e1 = 2 * i + 1 <= lim ? e1 : 0.f;
          }
          ls += e0 + e1;
          e0 *= wv;
          e1 *= wv;
          const __half2 hh = __floats2half2_rn(e0, e1);
          const float2 ff = __half22float2(hh);
          pk[i] = *reinterpret_cast<const uint32_t*>(&hh);
          pk[8 + i] = pack_f16(e0 - ff.x, e1 - ff.y);
        }
        l += ls;
        tmem_st16(ts + 16 * gi, pk);  // hi limbs in columns 0 .. 7 of the group's 16, lo limbs in 8 .. 15
      }
      // window tokens with infinities or NaN among their values lie as zeros in the tile, since zero weights
      // of rows that do not see them would not cancel them: the rows that do see them add them here
      float keep = av;
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) any |= sh.bad[st][i];
      if (any) {
#pragma unroll
        for (int i = 0; i < D; ++i) o[i] *= av;
        keep = 1.f;
#pragma unroll 1
        for (int t = 0; t < KT; ++t) {
          const int p = j * KT + t;
          if (!(sh.bad[st][t >> 4] >> (t & 15) & 1) || p > pos) continue;
          const size_t at = (((size_t)b * P.hkv + g) * C.ring + p % C.ring) * D;
          const long long qa = (((long long)b * n_query + rr / G) * P.hq + (long long)g * G + rr % G) * P.dh;
          float dot = 0.f;
#pragma unroll 1
          for (int i = 0; i < P.dh; ++i) dot = fmaf(load_elem(q, dtype, qa + i), __half2float(C.win_k[at + i]), dot);
          const float w = ex2(dot * (scale * kLog2e) - mb) * vi * kWeightTop;
#pragma unroll
          for (int i = 0; i < D; ++i) o[i] = fmaf(w, __half2float(C.win_v[at + i]), o[i]);
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_before();
      mbar_arrive(&sh.pready[u]);  // (nothing of the tile's scales is read after this)
      if (!mbar_wait(&sh.ofull[u], ph)) {
        failed = true;
        break;
      }
      tc_after();
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t v[16];
        tmem_ld16(to + 16 * c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[16 * c + i] = fmaf(o[16 * c + i], keep, __uint_as_float(v[i]));
      }
    }
    if (failed) {
      atomicOr(&g_int8_prefill_err, TQ_DEVERR_TIMEOUT);
      sh.fail = 1;
    }
    const float unit = vref * (1.f / kWeightTop);
#pragma unroll
    for (int i = 0; i < D; ++i) o[i] *= unit;
    if (RT == 1) {
      // the units meet: unit 1 leaves its rows in the (now idle) operand memory, column by column
      float* box = reinterpret_cast<float*>(smem + kSmemK);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (u == 1) {
#pragma unroll
        for (int i = 0; i < D; ++i) box[i * 128 + r] = o[i];
        sh.m[r] = m;
        sh.l[r] = l;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (u == 0) {
        const float m1 = sh.m[r], mn = fmaxf(m, m1), mb = mn == -INFINITY ? 0.f : mn;
        const float f0 = ex2(m - mb), f1 = ex2(m1 - mb);
        l = l * f0 + sh.l[r] * f1;
        m = mn;
#pragma unroll
        for (int i = 0; i < D; ++i) o[i] = o[i] * f0 + box[i * 128 + r] * f1;
      }
    }
    if ((RT == 2 || u == 0) && rr < rows) {
      const size_t head = ((size_t)b * n_query + rr / G) * P.hq + (size_t)g * G + rr % G;
      if (S == 1) {
        const float z = l == 0.f ? 0.f : 1.f / l;
        float* dst = out + head * P.dh;
#pragma unroll
        for (int i = 0; i < D; i += 4)
          if (i < P.dh) *reinterpret_cast<float4*>(dst + i) = make_float4(o[i] * z, o[i + 1] * z, o[i + 2] * z, o[i + 3] * z);
        if (lse) lse[head] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
      } else {
        float* dst = reinterpret_cast<float*>(ws + L.acc) + (head * S + split) * D;
#pragma unroll
        for (int i = 0; i < D; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        float* ml = reinterpret_cast<float*>(ws + L.ml) + (head * S + split) * 2;
        ml[0] = m * 0.6931471805599453f;  // the joining kernel takes natural logarithms
        ml[1] = l;
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ operands: groups cw and cw + 4 of every tile
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    const int cw = warp - 8, g8 = lane >> 2, t4 = lane & 3;
    uint4 kr[2][4], vr[2][4];
    const unsigned char* sb[2];
    float2 sc[2];
    // page of group x (0, 1) of tile j: its sub-block, or null
    auto page_of = [&](int j, int x) -> const unsigned char* {
      const int p0 = j * KT + (cw + 4 * x) * kPage;
      if (j >= j1 || p0 >= min(nc, end)) return nullptr;
      const long long page = C.block_table[(size_t)b * C.max_pages + p0 / kPage];
      if (page < 0 || page >= C.n_pages) {
        if (lane == 0) atomicOr(&g_int8_prefill_err, TQ_DEVERR_PAGE_INDEX);
        return nullptr;
      }
      return i8_subblock(P, C, page, g);
    };
    auto load_keys = [&](int j) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sb[x] = page_of(j, x);
        if (sb[x]) {
          sc[x] = *reinterpret_cast<const float2*>(sb[x] + i8_off_head(D));
#pragma unroll
          for (int i = 0; i < 4; ++i) kr[x][i] = *reinterpret_cast<const uint4*>(sb[x] + i8_off_kcodes(D) + i * 512 + lane * 16);
        }
      }
    };
    bool failed = false;
    load_keys(j0);
    for (int j = j0; j < j1; ++j) {
      const int st = (j - j0) & 1, sp = ((j - j0) >> 1) & 1;
      unsigned char* kt = smem + kSmemK + st * kKTile;
      unsigned char* vt = smem + kSmemV + st * kVTile;
      const unsigned char* cur[2] = {sb[0], sb[1]};
      const float2 csc[2] = {sc[0], sc[1]};
      if (!mbar_wait(&sh.kfree[st], sp ^ 1)) {
        failed = true;
        break;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int gi = cw + 4 * x, p0 = j * KT + gi * kPage;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int tok = 4 * (g8 >> 1) + 2 * nt + (g8 & 1), row = 16 * gi + tok;
          unsigned char* dst = kt + (row >> 3) * kKSbo + (row & 7) * 16 + 2 * t4 * kKLbo;
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            uint4 a = make_uint4(0, 0, 0, 0), c = a;
            if (cur[x]) {
              const uint4 w = kr[x][2 * nt + jj];
              a = make_uint4(i8_lo2(w.x), i8_hi2(w.x), i8_lo2(w.y), i8_hi2(w.y));
              c = make_uint4(i8_lo2(w.z), i8_hi2(w.z), i8_lo2(w.w), i8_hi2(w.w));
            } else if (p0 >= nc && p0 + tok < end) {
              const __half* rowp = C.win_k + (((size_t)b * P.hkv + g) * C.ring + (p0 + tok) % C.ring) * D + 64 * jj + 16 * t4;
              a = *reinterpret_cast<const uint4*>(rowp);
              c = *reinterpret_cast<const uint4*>(rowp + 8);
            }
            *reinterpret_cast<uint4*>(dst + 8 * jj * kKLbo) = a;
            *reinterpret_cast<uint4*>(dst + (8 * jj + 1) * kKLbo) = c;
          }
        }
        if (cur[x]) {  // the group's keys are on their way: its values take their registers
#pragma unroll
          for (int i = 0; i < 4; ++i) vr[x][i] = *reinterpret_cast<const uint4*>(cur[x] + i8_off_vcodes(D) + i * 512 + lane * 16);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.kfull[st]);
      load_keys(j + 1);
      if (!mbar_wait(&sh.vfree[st], sp ^ 1)) {
        failed = true;
        break;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int gi = cw + 4 * x, p0 = j * KT + gi * kPage;
        const bool win = !cur[x] && p0 >= nc && p0 < end;
        unsigned char* dst = vt + (2 * gi + (t4 >> 1)) * kVLbo + g8 * kVSbo + (t4 & 1) * 8;
        uint32_t bad = 0;
        if (!win) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // i = 2 jj + half
            uint4 w = vr[x][i];
            if (!cur[x]) w = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);  // codes 0
            unsigned char* d2 = dst + 8 * (i >> 1) * kVSbo + 64 * (i & 1);
            *reinterpret_cast<uint2*>(d2) = make_uint2(i8_lo2(w.x), i8_hi2(w.x));
            *reinterpret_cast<uint2*>(d2 + 16) = make_uint2(i8_lo2(w.y), i8_hi2(w.y));
            *reinterpret_cast<uint2*>(d2 + 32) = make_uint2(i8_lo2(w.z), i8_hi2(w.z));
            *reinterpret_cast<uint2*>(d2 + 48) = make_uint2(i8_lo2(w.w), i8_hi2(w.w));
          }
        } else {
          // four tokens' rows of 8 channels, twice; a token with a non-finite value anywhere is left out as a whole
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
            for (int jj = 0; jj < 2; ++jj) {
              uint32_t w[4][4];
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const int p = p0 + 4 * t4 + t;
                uint4 a = make_uint4(0, 0, 0, 0);
                if (p < end && !(pass && (bad >> (4 * t4 + t) & 1)))
                  a = *reinterpret_cast<const uint4*>(C.win_v + (((size_t)b * P.hkv + g) * C.ring + p % C.ring) * D + 64 * jj + 8 * g8);
                w[t][0] = a.x, w[t][1] = a.y, w[t][2] = a.z, w[t][3] = a.w;
                if (pass == 0) {
                  bool nf = false;
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    nf |= (w[t][e] & 0x7c00u) == 0x7c00u || (w[t][e] & 0x7c000000u) == 0x7c000000u;
                  if (nf) bad |= 1u << (4 * t4 + t);
                }
              }
              if (pass == 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
                  *reinterpret_cast<uint2*>(dst + 8 * jj * kVSbo + 16 * e) =
                      make_uint2(__byte_perm(w[0][e >> 1], w[1][e >> 1], sel), __byte_perm(w[2][e >> 1], w[3][e >> 1], sel));
                }
              }
            }
            if (pass == 0) bad = __reduce_or_sync(0xffffffffu, bad);
          }
        }
        if (lane == 0) {
          sh.scale[st][gi] = cur[x] ? csc[x] : make_float2(1.f, win ? 1.f : 0.f);
          sh.bad[st][gi] = bad;
          const bool there = cur[x] || win;
          if (there) atomicOr(&sh.live[st], 1u << gi);
          else atomicAnd(&sh.live[st], ~(1u << gi));
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.vfull[st]);
    }
    if (failed) {
      if (lane == 0) atomicOr(&g_int8_prefill_err, TQ_DEVERR_TIMEOUT);
      sh.fail = 1;
    }
  } else {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 12 && lane == 0 && j1 > j0) {
      const uint64_t dq = tc_desc(sbase + kSmemQ, kQLbo, kQSbo);
      bool ok = true;
      auto scores = [&](int u, int st) {  // S of unit u from the keys in stage st
        const uint64_t dk = tc_desc(sbase + kSmemK + st * kKTile, kKLbo, kKSbo);
#pragma unroll
        for (int ql = 0; ql < QL; ++ql) {
          const uint64_t da = dq + (uint64_t)(((RT == 2 ? u : ql) * kQTile) >> 4);
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tmem + 128u * u, da + (uint64_t)(2 * kQLbo >> 4) * k, dk + (uint64_t)(2 * kKLbo >> 4) * k, ql > 0 || k > 0);
        }
        tc_commit(&sh.sfull[u]);
      };
      auto values = [&](int u, int st) {  // O of unit u: 8 k-steps of 16 tokens, hi and lo limbs
        const uint64_t dv = tc_desc(sbase + kSmemV + st * kVTile, kVLbo, kVSbo);
        const uint32_t a = tmem + 128u * u, d = tmem + 256u + 128u * u;
#pragma unroll 1
        for (int k = 0; k < KT / 16; ++k) {
          mma_ts(d, a + 16u * k + 8u, dv + (uint64_t)(2 * kVLbo >> 4) * k, k > 0);
          mma_ts(d, a + 16u * k, dv + (uint64_t)(2 * kVLbo >> 4) * k, 1);
        }
        tc_commit(&sh.ofull[u]);
      };
      // tile of unit u's step i: RT = 2 both units take every tile, RT = 1 they take turns
      if (RT == 2) {
        ok = mbar_wait(&sh.kfull[0], 0);
        if (ok) {
          tc_after();
          scores(0, 0);
          scores(1, 0);
          tc_commit(&sh.kfree[0]);
        }
        for (int j = j0; ok && j < j1; ++j) {
          const int i = j - j0, st = i & 1, sp = (i >> 1) & 1, nst = (i + 1) & 1, nsp = ((i + 1) >> 1) & 1;
#pragma unroll 1
          for (int u = 0; ok && u < 2; ++u) {
            ok = mbar_wait(&sh.pready[u], i & 1) && mbar_wait(&sh.vfull[st], sp);
            if (!ok) break;
            tc_after();
            values(u, st);
            if (u == 1) tc_commit(&sh.vfree[st]);
            if (j + 1 < j1) {
              ok = mbar_wait(&sh.kfull[nst], nsp);
              if (!ok) break;
              tc_after();
              scores(u, nst);
              if (u == 1) tc_commit(&sh.kfree[nst]);
            }
          }
        }
      } else {
        for (int i = 0; ok && i < min(2, j1 - j0); ++i) {
          ok = mbar_wait(&sh.kfull[i], 0);
          if (!ok) break;
          tc_after();
          scores(i, i);
          tc_commit(&sh.kfree[i]);
        }
        for (int j = j0; ok && j < j1; ++j) {
          const int i = j - j0, u = i & 1, sp = (i >> 1) & 1;
          ok = mbar_wait(&sh.pready[u], sp) && mbar_wait(&sh.vfull[u], sp);
          if (!ok) break;
          tc_after();
          values(u, u);
          tc_commit(&sh.vfree[u]);
          if (j + 2 < j1) {
            ok = mbar_wait(&sh.kfull[u], sp ^ 1);
            if (!ok) break;
            tc_after();
            scores(u, u);
            tc_commit(&sh.kfree[u]);
          }
        }
      }
      // tensor memory is given back and the operands' memory reused only when every product has ended
      tc_commit(&sh.drained);
      if (!mbar_wait(&sh.drained, 0)) ok = false;
      if (!ok) {
        atomicOr(&g_int8_prefill_err, TQ_DEVERR_TIMEOUT);
        sh.fail = 1;
      }
    }
    __syncwarp();
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

}  // namespace

// Rows of a block's query tile: two tiles of 128.
bool int8_prefill_tc_ok(const KParams& P, int n_query) { return P.d == D && (long long)n_query * P.G > 16; }

// Splits of the key tiles: blocks are one to an SM, so the count whose last wave is fullest, at least four tiles
// a split; the joining costs a pass over the partial outputs (about 3 % of a block's work a split).
WsLayout int8_prefill_layout(const KParams& P, int batch, int n_query, int max_ctx, int num_sms) {
  const long long rt = ((long long)n_query * P.G + 255) / 256, units = std::max(1LL, rt * batch * P.hkv);
  const int tiles = std::max(1, (max_ctx + KT - 1) / KT);
  int best = 1;
  double best_eff = -1.0;
  for (int S = 1; S <= 64; ++S) {
    if (S > 1 && tiles / S < 4) break;
    if (units * S > 65535) break;
    const double w = (double)(units * S) / std::max(1, num_sms);
    const double eff = w / ceil(w) / (1.0 + 0.03 * (S - 1));
    if (eff > best_eff + 1e-9) {
      best_eff = eff;
      best = S;
    }
  }
  WsLayout L{};
  L.n_comp_splits = best;
  const size_t heads = (size_t)batch * n_query * P.hq;
  size_t o = 0;
  if (best > 1) {
    L.ml = o;
    o += (heads * best * 2 * sizeof(float) + 255) & ~(size_t)255;
    L.acc = o;
    o += (heads * best * (size_t)D * sizeof(float) + 255) & ~(size_t)255;
  }
  L.total = std::max<size_t>(o, 256);
  return L;
}

cudaError_t launch_int8_prefill(const KParams& P, const KCache& C, int n_query, const void* q, int dtype, float scale,
                                float* out, float* lse, void* ws, const WsLayout& L, int max_ctx, cudaStream_t st) {
  const int rows = n_query * P.G;
  unsigned char* w = reinterpret_cast<unsigned char*>(ws);
  // float queries take two limbs; a single tile of rows is split over the units by key tiles instead
  const bool one = dtype == TQ_F32 || rows <= 128;
  auto kern = dtype == TQ_F32 ? i8_prefill_attn_kernel<1, 2> : rows <= 128 ? i8_prefill_attn_kernel<1, 1> : i8_prefill_attn_kernel<2, 1>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  const int per = one ? 128 : 256;
  kern<<<dim3((rows + per - 1) / per, P.hkv, C.batch * L.n_comp_splits), kThreads, kSmemBytes, st>>>(P, C, n_query, q, dtype, scale,
                                                                                                 out, lse, w, L, max_ctx);
  if ((e = cudaGetLastError()) != cudaSuccess || L.n_comp_splits == 1) return e;
  return launch_int8_combine(P, w, L, (long long)C.batch * n_query, out, lse, st);
}

cudaError_t read_clear_int8_prefill_error(unsigned* bits) {
  unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_int8_prefill_err, sizeof(unsigned));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_int8_prefill_err, &zero, sizeof(unsigned));
}

}  // namespace tq
