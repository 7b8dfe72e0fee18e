// Attention over the 8-bit paged key/value cache, tiled kernel: prompts.
//
// Rows (new tokens x the query heads that share a key head) are taken R = 256
// (or 128) at a time as one or two tiles of 128; a step is 128 keys, two
// pages:   S = Q K^T (tcgen05, 128 x 128 x D),  weights,  O += P V (tcgen05,
// 128 x D x 128), with S, P and O in tensor memory.  Q is fp16 after an exact
// scaling of each row by a power of two (fp32 queries: the sum of two fp16
// parts), K and V are e4m3 widened exactly to fp16, P is fp16 (two parts for
// fp32 outputs); sums, maxima and the accumulators are fp32.
//
// The scale of a page's keys multiplies its logits.  The scale of its values
// goes into the weights, w = 2^(s - M + lv - LV) with lv = log2(v_scale) and
// LV the unit that O is held in, so O needs no scaling per page; the softmax
// sum takes w 2^(LV - lv).  When a page's lv is more than 3 away from LV, O
// is multiplied (fp32) into the unit of that page, and pages whose scales are
// further apart than that are never put into one step: a weight that fp16
// cannot hold is below 2^-29 of its row's largest, whatever the scales.  M is
// raised only when a row's maximum has grown by more than 2^4 since it was
// set, so that O is seldom rescaled; weights carry a factor 2^8.
//
// Roles (512 threads, one CTA per SM): warps 0-3 and 4-7 the softmax of tile
// 0 and 1 (a thread per row, no exchange between threads), warps 8-11 widen
// the pages from global memory into the swizzled operands, warp 12 issues
// every MMA, warp 13 walks the work list and looks up pages and scales.  The
// two tiles alternate: while one tile's softmax runs, the other's products do.
// Bound: the tensor cores, 4 D flops per visible (query head, key); next
// shared memory (operands of S from both tiles, the widened pages' writes).
//
// Work split: the steps of all (sequence, head, row tile) items form one
// list, cut into equal shares as in the streaming kernel; what a tile cannot
// see is not in the list.  Rows of a cut item leave fp32 partials that a
// second launch joins.
//
// Every wait is bounded (about one second): a timeout is recorded, all roles
// stop, the MMAs in flight are waited for and the tensor memory is freed.
#include <climits>

#include "np_kv.cuh"
#include "np_tc.cuh"

namespace np {

namespace {

constexpr int kTileThreads = 512;
constexpr int kMetaSlots = 8;
constexpr int kStepKeys = 128;
// log2 of: the growth a weight may show before M is raised, the distance of a
// page's value scale from O's unit, the factor on all weights.  Together they
// stay below fp16's largest, 2^16.
constexpr float kLazy = 4.f, kUnit = 3.f, kLift = 8.f;
constexpr int kCutCost = 8;    // steps that cutting an item costs (partials, second launch)

// NX tiles of 128 rows, NP fp16 parts of Q and P, NB operand buffers.
template <typename T, int D> struct TileShape {
  static constexpr int NP = sizeof(T) == 4 ? 2 : 1;
  static constexpr int NX = (D == 256 || NP == 2) ? 1 : 2;
  static constexpr int NB = D == 256 ? 1 : 2;
  static constexpr int R = 128 * NX;
  static constexpr uint32_t kQ = 128 * D * 2;            // bytes of one part of one tile's Q
  static constexpr uint32_t kKV = kStepKeys * D * 2;     // bytes of one operand buffer
  static constexpr uint32_t kOperands = NX * NP * kQ + 2 * NB * kKV;
  // tensor memory columns
  static constexpr uint32_t S(int x) { return x * 128u; }
  static constexpr uint32_t P(int x) { return NX == 2 ? x * 128u : 128u; }
  static constexpr uint32_t O(int x) { return 256u + x * (uint32_t)D; }
};

struct TileSeq {
  int row, begin, n, len;
};

struct TilePlan {
  long long chunk, total;
  int split;
};

// Keys that a tile's rows see, as a list of pages: slots [0, sink), [lo, ..).
struct TileKeys {
  int sink, lo, pages, p_min, p_max, rows;
  __device__ __forceinline__ int slot(int k) const { return k < sink ? k : lo + (k - sink); }
  __device__ __forceinline__ int steps() const { return (pages + 1) >> 1; }
};

template <int R>
__device__ __forceinline__ TileKeys tile_keys(const KvAttend& a, int n, int len, int tile) {
  const int g = a.Hq / a.kv.H;
  const long long all = n * (long long)g, first = (long long)tile * R;
  TileKeys t;
  t.rows = (int)(all - first < R ? all - first : R);
  t.p_min = len - n + (int)(first / g);
  t.p_max = len - n + (int)((first + t.rows - 1) / g);
  if (t.p_min < -1) t.p_min = -1;
  if (t.p_max < -1) t.p_max = -1;
  const int hi = t.p_max >= 0 ? t.p_max / kKvPage + 1 : 0;
  t.lo = t.sink = 0;
  if (a.window > 0) {
    const long long low = (long long)t.p_min - a.window + 1;
    t.lo = low > 0 ? (int)(low / kKvPage) : 0;
    const int s = a.sinks / kKvPage + (a.sinks % kKvPage != 0);
    t.sink = s < t.lo ? s : t.lo;
  }
  t.pages = t.sink + hi - t.lo;
  if (t.pages < 1) t.pages = 1;  // an item without keys still writes its zeros
  return t;
}

__device__ __forceinline__ int tiles_of(const KvAttend& a, int n, int R) {
  return (int)((n * (long long)(a.Hq / a.kv.H) + R - 1) / R);
}

// Numbers the units (steps, or whole items where nothing is to be gained by
// cutting): pre[i] = units before sequence i; per[i] = units of one head of
// sequence i.  Called by the whole CTA.
template <int R>
__device__ __forceinline__ TilePlan tile_plan(const KvAttend& a, int ctas, long long* pre, int* per, TileSeq* seq,
                                              long long* tmp) {
  const int n = a.batch.n_seqs;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const KvSeq s = kv_seq(a.kv, a.batch, i);
    seq[i] = TileSeq{s.row, s.begin, s.n, s.len};
  }
  if (threadIdx.x == 0) tmp[2] = 0;
  __syncthreads();
  for (int i = warp; i < n; i += warps) {
    const int tiles = tiles_of(a, seq[i].n, R);
    int steps = 0, longest = 0;
    for (int t = lane; t < tiles; t += 32) {
      const int s = tile_keys<R>(a, seq[i].n, seq[i].len, t).steps();
      steps += s;
      longest = s > longest ? s : longest;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      steps += __shfl_xor_sync(0xffffffffu, steps, o);
      const int l = __shfl_xor_sync(0xffffffffu, longest, o);
      longest = l > longest ? l : longest;
    }
    if (lane == 0) {
      per[i] = steps;
      atomicMax(reinterpret_cast<unsigned long long*>(&tmp[2]), (unsigned long long)longest);
    }
  }
  __syncthreads();
  if (warp == 0) {
    long long items = 0, steps = 0;
    for (int i = lane; i < n; i += 32) {
      items += (long long)tiles_of(a, seq[i].n, R) * a.kv.H;
      steps += (long long)per[i] * a.kv.H;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      items += __shfl_xor_sync(0xffffffffu, items, o);
      steps += __shfl_xor_sync(0xffffffffu, steps, o);
    }
    const bool split = (items + ctas - 1) / ctas * tmp[2] > steps / ctas + kCutCost;
    long long run = 0;
    for (int base = 0; base < n; base += 32) {
      const int i = base + lane;
      long long u = 0;
      if (i < n) {
        if (!split) per[i] = tiles_of(a, seq[i].n, R);
        u = (long long)per[i] * a.kv.H;
      }
      long long x = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (i < n) pre[i] = run + x - u;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      pre[n] = run;
      tmp[0] = (run + ctas - 1) / ctas;
      tmp[1] = split;
    }
  }
  __syncthreads();
  TilePlan p;
  p.chunk = tmp[0] > 0 ? tmp[0] : 1;
  p.total = pre[n];
  p.split = (int)tmp[1];
  return p;
}

// A place in the list of units.
struct TilePos {
  int b, h, tile;
  int step;  // step of the item (0 where units are items)
  int tiles;
};

// Unit u (called by a whole warp).
template <int R>
__device__ __forceinline__ TilePos tile_find(const KvAttend& a, const TilePlan& p, const long long* pre,
                                             const int* per, const TileSeq* seq, long long u) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.batch.n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= u) lo = mid; else hi = mid;
  }
  TilePos t;
  t.b = lo;
  t.tiles = tiles_of(a, seq[lo].n, R);
  const long long off = u - pre[lo];
  t.h = (int)(off / per[lo]);
  int rem = (int)(off % per[lo]);
  t.step = 0;
  t.tile = rem;
  if (!p.split) return t;
  for (int base = 0; base < t.tiles; base += 32) {
    const int i = base + lane;
    const int s = i < t.tiles ? tile_keys<R>(a, seq[lo].n, seq[lo].len, i).steps() : 0;
    int x = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, x > rem);
    if (hit) {
      const int l = __ffs(hit) - 1;
      t.tile = base + l;
      t.step = rem - __shfl_sync(0xffffffffu, x - s, l);
      return t;
    }
    rem -= __shfl_sync(0xffffffffu, x, 31);
  }
  t.tile = t.tiles - 1;  // not reached: rem < per[lo]
  return t;
}

struct StepMeta {
  int flags;     // 1: first of a stretch, 2: last, 4: no more work, 8: stretch starts its item, 16: ends it
  int nx;        // tiles with rows
  int page[2];   // -1: nothing
  int base[2];   // position of the first token
  float ks[2], lv[2];  // key scale, log2 of the value scale
  int row0;      // first row of the item in its sequence and head
  int rows;
  int begin, n, len, h;
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] x B[smem]^T, issued by one thread.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t no_nan(uint32_t v) {
  const __half2 h = __hmin2(*reinterpret_cast<__half2*>(&v), __floats2half2_rn(448.f, 448.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes of T from floats.
template <typename T> __device__ __forceinline__ uint4 pack_chunk(const float* f);
template <> __device__ __forceinline__ uint4 pack_chunk<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <> __device__ __forceinline__ uint4 pack_chunk<__half>(const float* f) {
  return make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
}
template <> __device__ __forceinline__ uint4 pack_chunk<__nv_bfloat16>(const float* f) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// 16 codes as 16 fp16 values into two 16-byte chunks.
template <bool CLEAN>
__device__ __forceinline__ void widen16(const uint4& v, uint32_t a0, uint32_t a1) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = e4m3x2_to_f16x2(w[i] & 0xffffu);
    f[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
  }
  if constexpr (CLEAN) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = no_nan(f[i]);
  }
  sts128(a0, f[0], f[1], f[2], f[3]);
  sts128(a1, f[4], f[5], f[6], f[7]);
}

struct TileShared {
  uint64_t meta_full[kMetaSlots], meta_empty[kMetaSlots];
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t qready[2], sfull[2], pready[2], pvdone[2], drained;
  StepMeta meta[kMetaSlots];
  long long tmp[3];
  uint32_t tmem;
  int abort;
};

template <int D, int R> struct TilePartial {
  static constexpr size_t kFloats = (size_t)R * (D + 2);
  __device__ static float* o(void* ws, int slot) { return static_cast<float*>(ws) + slot * kFloats; }
  __device__ static float* m(void* ws, int slot) { return o(ws, slot) + R * D; }
  __device__ static float* l(void* ws, int slot) { return o(ws, slot) + R * D + R; }
};

template <typename T, int D>
__global__ void __launch_bounds__(kTileThreads, 1) attend_tile_kernel(const KvAttend a) {
  using Sh = TileShape<T, D>;
  constexpr int NX = Sh::NX, NP = Sh::NP, NB = Sh::NB, R = Sh::R;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ TileShared sh;

  uint8_t* ops = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t q_s = smem_addr(ops), k_s = q_s + NX * NP * Sh::kQ, v_s = k_s + NB * Sh::kKV;
  long long* pre = reinterpret_cast<long long*>(ops + Sh::kOperands);
  TileSeq* seq = reinterpret_cast<TileSeq*>(pre + a.batch.n_seqs + 1 + ((a.batch.n_seqs + 1) & 1));
  int* per = reinterpret_cast<int*>(seq + a.batch.n_seqs);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kMetaSlots; ++i) {
      mbar_init(&sh.meta_full[i], 1);
      mbar_init(&sh.meta_empty[i], 4 * NX + 4 + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.kfull[i], 4);
      mbar_init(&sh.kempty[i], 1);
      mbar_init(&sh.vfull[i], 4);
      mbar_init(&sh.vempty[i], 1);
      mbar_init(&sh.qready[i], 4);
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pready[i], 4);
      mbar_init(&sh.pvdone[i], 1);
    }
    mbar_init(&sh.drained, 1);
    sh.abort = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_addr(&sh.tmem), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  const TilePlan p = tile_plan<R>(a, gridDim.x, pre, per, seq, sh.tmp);  // synchronises the CTA
  tc_fence_after();
  grid_dependents_launch();
  const uint32_t tmem = sh.tmem;
  const int g = a.Hq / a.kv.H;
  volatile int* abort = &sh.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_phase(smem_addr(bar), parity, abort, a.kv.err); };

  if (warp == 13) {
    // ---- work list ----
    const long long u0 = (long long)blockIdx.x * p.chunk;
    const long long u1 = u0 + p.chunk < p.total ? u0 + p.chunk : p.total;
    uint32_t count = 0;
    bool alive = true;
    // the next free slot of the list (all lanes)
    auto slot_free = [&]() {
      if (count >= kMetaSlots)
        alive = alive && wait(&sh.meta_empty[count % kMetaSlots], (count / kMetaSlots - 1) & 1);
      alive = __all_sync(0xffffffffu, alive);
      return alive;
    };
    if (u0 < u1) {
      TilePos t = tile_find<R>(a, p, pre, per, seq, u0);
      for (long long u = u0; u < u1 && alive;) {
        const TileSeq w = seq[t.b];
        const TileKeys tk = tile_keys<R>(a, w.n, w.len, t.tile);
        const int steps = tk.steps();
        const int s0 = t.step;
        int s1 = steps;
        if (p.split && (long long)(steps - s0) > u1 - u) s1 = s0 + (int)(u1 - u);
        for (int sb = s0; sb < s1 && alive; sb += 16) {
          // lane = page: the entries and scales of 16 steps at a time
          const int k = 2 * sb + lane;
          int page = -1, base = -1;
          float ks = 0.f, vs = 1.f;
          if (k < tk.pages && k < 2 * s1) {
            const int slot = tk.slot(k);
            if (slot * kKvPage <= tk.p_max) {
              page = a.kv.table[(size_t)w.row * a.kv.max_pages + slot];
              if (page < 0 || page >= a.kv.n_pages) {
                if (page != -1) atomicExch(a.kv.err, kDevErrBounds);
                page = -1;
              } else {
                base = slot * kKvPage;
                ks = a.kv.k_scale[(size_t)page * a.kv.H + t.h];
                vs = a.kv.v_scale[(size_t)page * a.kv.H + t.h];
                vs = fminf(fmaxf(vs, 9.094947017729282e-13f), 1099511627776.f);  // 2^-40, 2^40
              }
            }
          }
          // exact where the scale is a power of two
          const uint32_t vu = __float_as_uint(vs);
          const float lv = (vu & 0x7fffffu) == 0 ? (float)((int)(vu >> 23) - 127) : log2f(vs);
          // steps whose two pages have scales too far apart become two
          const float other = __shfl_xor_sync(0xffffffffu, lv, 1);
          const int mate = __shfl_xor_sync(0xffffffffu, page, 1);
          const unsigned apart = __ballot_sync(0xffffffffu, page >= 0 && mate >= 0 && fabsf(lv - other) > kUnit);
          for (int i = 0; i < 16 && sb + i < s1; ++i) {
            const int parts = (apart >> (2 * i)) & 1 ? 2 : 1;
            for (int part = 0; part < parts; ++part) {
              if (!slot_free()) break;
              StepMeta* m = &sh.meta[count % kMetaSlots];
              if ((lane >> 1) == i) {
                const int x = lane & 1;
                const bool here = parts == 1 || x == part;
                m->page[x] = here ? page : -1;
                m->base[x] = here ? base : -1;
                m->ks[x] = ks;
                m->lv[x] = lv;
              }
              if (lane == 0) {
                const int s = sb + i;
                m->flags = (s == s0 && part == 0 ? 1 : 0) | (s == s1 - 1 && part == parts - 1 ? 2 : 0) |
                           (s0 == 0 ? 8 : 0) | (s1 == steps ? 16 : 0);
                m->nx = (tk.rows + 127) / 128;
                m->row0 = t.tile * R;
                m->rows = tk.rows;
                m->begin = w.begin;
                m->n = w.n;
                m->len = w.len;
                m->h = t.h;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive_local(smem_addr(&sh.meta_full[count % kMetaSlots]));
              ++count;
            }
          }
        }
        u += p.split ? s1 - s0 : 1;
        // the next item
        t.step = 0;
        if (++t.tile == t.tiles) {
          t.tile = 0;
          if (++t.h == a.kv.H) {
            t.h = 0;
            do {
              ++t.b;
              t.tiles = t.b < a.batch.n_seqs ? tiles_of(a, seq[t.b].n, R) : 1;
            } while (t.tiles == 0);
          }
        }
      }
    }
    if (slot_free()) {
      if (lane == 0) {
        sh.meta[count % kMetaSlots].flags = 4;
        mbar_arrive_local(smem_addr(&sh.meta_full[count % kMetaSlots]));
      }
    }
  } else if (warp == 12) {
    // ---- MMA issue: one thread ----
    if (lane == 0) {
      constexpr uint32_t id_qk = idesc_f16(false, false, 128, kStepKeys);
      constexpr uint32_t id_pv = idesc_f16(false, false, 128, D);
      uint32_t mcount = 0, n_pv[2] = {0, 0}, n_q[2] = {0, 0}, steps = 0;
      int flags = 4, nx = 0;
      auto next_meta = [&](int& f, int& x) {
        const uint32_t st = mcount % kMetaSlots;
        if (!wait(&sh.meta_full[st], (mcount / kMetaSlots) & 1)) return false;
        f = sh.meta[st].flags;
        x = sh.meta[st].nx;
        mbar_arrive_local(smem_addr(&sh.meta_empty[st]));
        ++mcount;
        return true;
      };
      // S of tile x for step `i` (of this CTA)
      auto issue_qk = [&](int x, uint32_t i, bool first, bool last_tile) {
        const uint32_t kb = i % NB;
        if (x == 0 && !wait(&sh.kfull[kb], (i / NB) & 1)) return false;
        if (n_pv[x] && !wait(&sh.pvdone[x], (n_pv[x] - 1) & 1)) return false;
        if (first && !wait(&sh.qready[x], n_q[x]++ & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int pt = 0; pt < NP; ++pt)
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * 16384u + (k & 3) * 32u;
            tc_mma(tmem + Sh::S(x), smem_desc_sw128(q_s + (x * NP + pt) * Sh::kQ + off, 0, 1024),
                   smem_desc_sw128(k_s + kb * Sh::kKV + off, 0, 1024), id_qk, pt || k);
          }
        tc_commit(smem_addr(&sh.sfull[x]));
        if (last_tile) tc_commit(smem_addr(&sh.kempty[kb]));
        return true;
      };
      auto issue_pv = [&](int x, uint32_t i, bool first, bool last_tile) {
        const uint32_t vb = i % NB;
        if (x == 0 && !wait(&sh.vfull[vb], (i / NB) & 1)) return false;
        if (!wait(&sh.pready[x], n_pv[x] & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int pt = 0; pt < NP; ++pt)
#pragma unroll
          for (int k = 0; k < kStepKeys / 16; ++k)
            tc_mma_ts(tmem + Sh::O(x), tmem + Sh::P(x) + pt * 64 + k * 8,
                      smem_desc_sw128(v_s + vb * Sh::kKV + (k >> 2) * (D * 128u) + (k & 3) * 32u, 0, 1024), id_pv,
                      !first || pt || k);
        tc_commit(smem_addr(&sh.pvdone[x]));
        if (last_tile) tc_commit(smem_addr(&sh.vempty[vb]));
        ++n_pv[x];
        return true;
      };
      bool ok = next_meta(flags, nx);
      if (ok && !(flags & 4))
        for (int x = 0; x < nx && ok; ++x) ok = issue_qk(x, 0, true, x == nx - 1);
      while (ok && !(flags & 4)) {
        int nf = 4, nnx = 0;
        ok = next_meta(nf, nnx);
        if (!ok) break;
        const bool more = !(nf & 4), fresh = (nf & 1) != 0;
        if (more && !fresh) {
          for (int x = 0; x < nx && ok; ++x) {
            ok = issue_pv(x, steps, flags & 1, x == nx - 1);
            if (ok) ok = issue_qk(x, steps + 1, false, x == nx - 1);
          }
        } else {
          // a stretch ends here: both tiles' products first, since the next
          // stretch's queries come only after their results were taken
          for (int x = 0; x < nx && ok; ++x) ok = issue_pv(x, steps, flags & 1, x == nx - 1);
          if (more)
            for (int x = 0; x < nnx && ok; ++x) ok = issue_qk(x, steps + 1, true, x == nnx - 1);
        }
        flags = nf;
        nx = nnx;
        ++steps;
      }
      // nothing of this CTA may be in flight when it frees the tensor memory
      tc_commit(smem_addr(&sh.drained));
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&sh.drained, 0))
        if (global_ns() - t0 > kWaitLimitNs) break;
    }
    __syncwarp();
  } else if (warp >= 8 && warp < 12) {
    // ---- widening: units K(0), V(0), K(1), V(1), .. ----
    const int ct = tid - 256;
    constexpr int CH = D / 16;                       // 16-byte chunks of a token's keys
    constexpr int PER_PAGE = kKvPage * CH / 128;     // chunks per thread of one page
    constexpr int NC = D == 256 ? PER_PAGE : 2 * PER_PAGE;  // chunks in flight per thread
    constexpr int PIECES = 2 * PER_PAGE / NC;
    // place of a thread's c-th chunk of a page: eight neighbouring lanes hold
    // two rows x four chunks, whose fp16 images meet no bank twice
    const int qd = lane >> 3, l8 = lane & 7;
    const int k_ch = (qd % (D / 64)) * 4 + (l8 & 3), k_tok = (qd / (D / 64)) * 2 + (l8 >> 2);
    const int cw = ct >> 5;
    constexpr int TOK_W = 32 / CH;                   // tokens per warp and chunk index
    uint4 buf[NC];
    auto load = [&](const StepMeta& m, int side, int piece) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int all = piece * NC + c, half = all / PER_PAGE, i = all % PER_PAGE;
        const int page = m.page[half];
        uint4 v = make_uint4(0, 0, 0, 0);
        if (page >= 0) {
          const size_t block = (size_t)page * a.kv.H + m.h;
          const uint8_t* src = (side ? a.kv.v : a.kv.k) + block * kKvPage * D;
          src += side ? (i * 128 + ct) * 16 : ((i * 4 + cw) * TOK_W + k_tok) * D + k_ch * 16;
          v = *reinterpret_cast<const uint4*>(src);
        }
        buf[c] = v;
      }
    };
    auto store = [&](uint32_t dst, int side, int piece, int tail) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int all = piece * NC + c, half = all / PER_PAGE, i = all % PER_PAGE;
        if (side == 0) {
          const int t = half * kKvPage + (i * 4 + cw) * TOK_W + k_tok;
          const uint32_t row = dst + (k_ch >> 2) * 16384u + t * 128u;
          const int ck = (k_ch & 3) * 2;
          widen16<false>(buf[c], row + ((ck ^ (t & 7)) << 4), row + (((ck + 1) ^ (t & 7)) << 4));
        } else {
          const int d = (i * 128 + ct) >> 2, ck = ((i * 128 + ct) & 3) * 2;
          const uint32_t row = dst + half * (D * 128u) + d * 128u;
          const uint32_t a0 = row + ((ck ^ (d & 7)) << 4), a1 = row + (((ck + 1) ^ (d & 7)) << 4);
          if (tail) widen16<true>(buf[c], a0, a1);  // bytes behind the end may be NaN
          else widen16<false>(buf[c], a0, a1);
        }
      }
    };
    bool alive = true;
    auto read_meta = [&](uint32_t i, StepMeta& m) {
      const uint32_t st = i % kMetaSlots;
      alive = alive && wait(&sh.meta_full[st], (i / kMetaSlots) & 1);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) return false;
      m.flags = sh.meta[st].flags;
      m.page[0] = sh.meta[st].page[0];
      m.page[1] = sh.meta[st].page[1];
      m.base[0] = sh.meta[st].base[0];
      m.base[1] = sh.meta[st].base[1];
      m.h = sh.meta[st].h;
      m.len = sh.meta[st].len;
      __syncwarp();
      if (lane == 0) mbar_arrive_local(smem_addr(&sh.meta_empty[st]));
      return (m.flags & 4) == 0;
    };
    StepMeta m{};
    bool any = read_meta(0, m);
    if (any) load(m, 0, 0);
    for (uint32_t i = 0; any; ++i) {
      StepMeta nm{};
      bool more = false;
      const uint32_t b = i % NB;
      const int tail = m.base[0] + kKvPage > m.len || m.base[1] + kKvPage > m.len;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        uint64_t* empty = side ? &sh.vempty[b] : &sh.kempty[b];
        if (i >= NB) alive = alive && wait(empty, (i / NB - 1) & 1);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;
#pragma unroll
        for (int piece = 0; piece < PIECES; ++piece) {
          store((side ? v_s : k_s) + b * Sh::kKV, side, piece, tail);
          // the next piece's codes are on their way while the others work
          if (piece + 1 < PIECES) load(m, side, piece + 1);
          else if (side == 0) load(m, 1, 0);
          else {
            more = read_meta(i + 1, nm);
            if (more) load(nm, 0, 0);
          }
        }
        fence_proxy_async_cta();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(smem_addr(side ? &sh.vfull[b] : &sh.kfull[b]));
      }
      if (!alive) break;
      m = nm;
      any = more;
    }
  } else if (warp < 4 * NX) {
    // ---- softmax: a thread per row ----
    const int X = warp >> 2;
    const int row = tid & 127;                             // row of the tile = lane of tensor memory
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // (32 * warp) << 16
    const uint32_t t_s = lanes + Sh::S(X), t_p = lanes + Sh::P(X), t_o = lanes + Sh::O(X);
    uint32_t mcount = 0, n_steps = 0;
    float ref = -INFINITY, l = 0.f, fac = 0.f;
    float unit = 0.f;       // log2 of the unit of O
    bool has_unit = false;
    int pos = -1;
    bool alive = true;
    for (;;) {
      const uint32_t st = mcount % kMetaSlots;
      alive = wait(&sh.meta_full[st], (mcount / kMetaSlots) & 1);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) break;
      const StepMeta m = sh.meta[st];
      __syncwarp();
      if (lane == 0) mbar_arrive_local(smem_addr(&sh.meta_empty[st]));
      ++mcount;
      if (m.flags & 4) break;
      if (X >= m.nx) continue;
      const int at = m.row0 + X * 128 + row;               // row of the sequence and head
      const bool in = X * 128 + row < m.rows;
      const int tok = at / g, head = m.h * g + at % g;
      if (m.flags & 1) {
        // this row's query, scaled so that its largest element is in [2^14, 2^15)
        const T* q = static_cast<const T*>(a.q) + (long long)(m.begin + tok) * a.q_tok + (long long)head * a.q_head;
        const bool wide_ok = (reinterpret_cast<uintptr_t>(q) & 15) == 0;
        float top = 0.f;
        constexpr int E = Elem<T>::E;
        for (int pass = 0; pass < 2; ++pass) {
          float up = 1.f;
          if (pass) {
            int e = (int)(__float_as_uint(top) >> 23) - 127;
            e = e < -112 ? -112 : e;
            up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
            fac = __uint_as_float((uint32_t)(e - 14 + 127) << 23) * a.scale_log2;
          }
#pragma unroll 2
          for (int d = 0; d < D; d += 8) {
            float x[8];
            if (!in) {
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = 0.f;
            } else if (wide_ok) {
#pragma unroll
              for (int i = 0; i < 8 / E; ++i)
                Elem<T>::load(*reinterpret_cast<const uint4*>(q + d + i * E), x + i * E);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = kv_to_float<T>(q[d + i]);
            }
            if (!pass) {
#pragma unroll
              for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
            } else {
              uint32_t h[4], lo[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x0 = x[2 * i] * up, x1 = x[2 * i + 1] * up;
                h[i] = pack_f16(x0, x1);
                if constexpr (NP == 2) {
                  const float2 f = f16x2_to_f32x2(h[i]);
                  lo[i] = pack_f16(x0 - f.x, x1 - f.y);
                }
              }
              const uint32_t off = (d >> 6) * 16384u + row * 128u + ((((d & 63) >> 3) ^ (row & 7)) << 4);
              sts128(q_s + X * NP * Sh::kQ + off, h[0], h[1], h[2], h[3]);
              if constexpr (NP == 2) sts128(q_s + (X * NP + 1) * Sh::kQ + off, lo[0], lo[1], lo[2], lo[3]);
            }
          }
        }
        pos = m.len - m.n + tok;
        if (!in || pos < -1) pos = -1;
        ref = -INFINITY;
        l = 0.f;
        unit = 0.f;
        has_unit = false;
        fence_proxy_async_cta();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(smem_addr(&sh.qready[X]));
      }
      alive = wait(&sh.sfull[X], n_steps & 1);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) break;
      tc_fence_after();
      // keys of half h that this row sees: columns [from, to] and below `sink`
      const float f[2] = {fac * m.ks[0], fac * m.ks[1]};
      bool whole[2];
      int from[2], to[2], sink[2];
      const int low = a.window == 0 || a.window > pos ? 0 : pos - a.window + 1;
      const int w_min = __reduce_min_sync(0xffffffffu, in ? pos : INT_MAX), w_max = __reduce_max_sync(0xffffffffu, pos);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = m.base[h];
        whole[h] = b >= 0 && b + kKvPage - 1 <= w_min &&
                   (a.window == 0 || b > w_max - a.window || b + kKvPage - 1 < a.sinks);
        to[h] = b < 0 ? -1 : pos - b;
        from[h] = low - b;
        sink[h] = b < 0 ? 0 : a.sinks - b;
      }
      float top = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float t = -INFINITY;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float s[32];
          tmem_ld32(t_s + h * 64 + c, s);
          if (whole[h]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) t = fmaxf(t, s[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int k = c + i;
              if (k <= to[h] && (k >= from[h] || k < sink[h])) t = fmaxf(t, s[i]);
            }
          }
        }
        if (t != -INFINITY) top = fmaxf(top, t * f[h]);
        __syncwarp();
      }
      // raise the reference only when the weights would grow past 2^kLazy
      float alpha = 1.f;
      if (top > ref + kLazy || (ref == -INFINITY && top != -INFINITY)) {
        alpha = ex2(ref - top);  // 0 from -infinity
        ref = top;
        l *= alpha;
      }
      // O's unit (the same for every row)
      float most = -INFINITY, least = INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (m.base[h] >= 0) {
          most = fmaxf(most, m.lv[h]);
          least = fminf(least, m.lv[h]);
        }
      if (most != -INFINITY && (!has_unit || most - unit > kUnit || unit - least > kUnit)) {
        if (has_unit) alpha *= ex2(unit - most);
        unit = most;
        has_unit = true;
      }
      if (!(m.flags & 1) && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tmem_ld16(t_o + c, o);
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(o[i] * alpha);
          tmem_st16(t_o + c, r);
        }
      }
      const float zero = ref == -INFINITY ? 0.f : ref;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float shift = m.base[h] >= 0 ? m.lv[h] - unit : 0.f;
        const float add = shift - zero + kLift;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float s[32];
          tmem_ld32(t_s + h * 64 + c, s);
          if (whole[h]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = ex2(fmaf(s[i], f[h], add));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int k = c + i;
              const bool see = k <= to[h] && (k >= from[h] || k < sink[h]);
              s[i] = see ? ex2(fmaf(s[i], f[h], add)) : 0.f;
            }
          }
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            sum += s[2 * i] + s[2 * i + 1];
            r[i] = pack_f16(s[2 * i], s[2 * i + 1]);
          }
          tmem_st16(t_p + h * 32 + c / 2, r);
          if constexpr (NP == 2) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 b = f16x2_to_f32x2(r[i]);
              r[i] = pack_f16(s[2 * i] - b.x, s[2 * i + 1] - b.y);
            }
            tmem_st16(t_p + 64 + h * 32 + c / 2, r);
          }
        }
        l = fmaf(sum, ex2(-shift), l);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_local(smem_addr(&sh.pready[X]));
      ++n_steps;

      if (m.flags & 2) {
        alive = wait(&sh.pvdone[X], (n_steps - 1) & 1);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;
        tc_fence_after();
        const bool cut = (m.flags & 24) != 24;
        const int slot = 2 * blockIdx.x + ((m.flags & 8) ? 1 : 0);
        float* po = TilePartial<D, R>::o(a.ws, slot) + (size_t)(X * 128 + row) * D;
        T* out = static_cast<T*>(a.out) + (long long)(m.begin + tok) * a.o_tok + (long long)head * a.o_head;
        const bool wide_ok = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        const float back = ex2(unit);  // O in the values' own unit
        const float inv = l == 0.f ? 0.f : back / l;
        if (cut && in) {
          TilePartial<D, R>::m(a.ws, slot)[X * 128 + row] = ref;
          TilePartial<D, R>::l(a.ws, slot)[X * 128 + row] = l;
        }
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tmem_ld16(t_o + c, o);
          if (in) {
            if (cut) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(po + c + i) = make_float4(o[i] * back, o[i + 1] * back, o[i + 2] * back, o[i + 3] * back);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= inv;
              if (wide_ok) {
#pragma unroll
                for (int i = 0; i < 16; i += Elem<T>::E)
                  *reinterpret_cast<uint4*>(out + c + i) = pack_chunk<T>(o + i);
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) out[c + i] = kv_from_float<T>(o[i]);
              }
            }
          }
          __syncwarp();
        }
        tc_fence_before();  // before the next stretch's products overwrite O
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of items that were cut: CTA (c, y) rows 8 y .. 8 y + 7
// of the item that the cut in front of share c opens.
template <typename T, int D>
__global__ void __launch_bounds__(256) tile_join_kernel(const KvAttend a, int ctas) {
  constexpr int R = TileShape<T, D>::R;
  constexpr int V = D / 32;  // elements per lane
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ long long tmp[3];
  long long* pre = reinterpret_cast<long long*>(smem_raw);
  TileSeq* seq = reinterpret_cast<TileSeq*>(pre + a.batch.n_seqs + 1 + ((a.batch.n_seqs + 1) & 1));
  int* per = reinterpret_cast<int*>(seq + a.batch.n_seqs);
  const TilePlan p = tile_plan<R>(a, ctas, pre, per, seq, tmp);
  grid_dependency_wait();
  const long long u = (long long)blockIdx.x * p.chunk;
  if (!p.split || u >= p.total) return;
  const TilePos t = tile_find<R>(a, p, pre, per, seq, u);
  if (t.step == 0 || t.step > p.chunk) return;  // the cut lies between items, or not first in its item
  const TileSeq w = seq[t.b];
  const TileKeys tk = tile_keys<R>(a, w.n, w.len, t.tile);
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= tk.rows) return;
  const int more = (int)((tk.steps() - t.step + p.chunk - 1) / p.chunk);
  const int c0 = blockIdx.x - 1;
  float top = TilePartial<D, R>::m(a.ws, 2 * c0 + 1)[row];
  for (int i = 1; i <= more; ++i) top = fmaxf(top, TilePartial<D, R>::m(a.ws, 2 * (c0 + i))[row]);
  const float zero = top == -INFINITY ? 0.f : top;
  float sum = 0.f, y[V];
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = 0.f;
  for (int i = 0; i <= more; ++i) {
    const int slot = 2 * (c0 + i) + (i == 0 ? 1 : 0);
    const float f = ex2(TilePartial<D, R>::m(a.ws, slot)[row] - zero);
    sum = fmaf(TilePartial<D, R>::l(a.ws, slot)[row], f, sum);
    const float* o = TilePartial<D, R>::o(a.ws, slot) + (size_t)row * D + lane;
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = fmaf(o[32 * j], f, y[j]);
  }
  const int g = a.Hq / a.kv.H, at = t.tile * R + row;
  T* out = static_cast<T*>(a.out) + (long long)(w.begin + at / g) * a.o_tok + (long long)(t.h * g + at % g) * a.o_head;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int j = 0; j < V; ++j) out[lane + 32 * j] = kv_from_float<T>(y[j] * inv);
}

template <typename T, int D> struct TileTag {};

template <typename T, int D>
cudaError_t launch_tile(const KvAttend& a, cudaStream_t st) {
  using Sh = TileShape<T, D>;
  const int ctas = kv_attend_ctas();
  if (ctas < 1) return cudaErrorInvalidDevice;
  const size_t list = ((size_t)a.batch.n_seqs + 2) * 8 + (size_t)a.batch.n_seqs * (sizeof(TileSeq) + 4);
  const size_t smem = 1024 + Sh::kOperands + list;
  auto kern = attend_tile_kernel<T, D>;
  cudaError_t e = ensure_dyn_smem<TileTag<T, D>>(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kTileThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  PdlConfig pdl(dim3((unsigned)ctas, Sh::R / 8), dim3(256), list, st);
  return cudaLaunchKernelEx(&pdl.cfg, tile_join_kernel<T, D>, a, ctas);
}

}  // namespace

bool kv_tile_takes(int dtype, int head_dim) { return dtype != 0 || head_dim != 256; }

size_t kv_tile_workspace(int dtype, int head_dim) {
  const int rows = dtype == 0 || head_dim == 256 ? 128 : 256;
  return (size_t)2 * kv_attend_ctas() * rows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_tile(const KvAttend& a, cudaStream_t st) {
  switch (a.dtype) {
    case 0: return a.kv.D == 64 ? launch_tile<float, 64>(a, st) : launch_tile<float, 128>(a, st);
    case 1:
      return a.kv.D == 64    ? launch_tile<__half, 64>(a, st)
             : a.kv.D == 128 ? launch_tile<__half, 128>(a, st)
                             : launch_tile<__half, 256>(a, st);
    default:
      return a.kv.D == 64    ? launch_tile<__nv_bfloat16, 64>(a, st)
             : a.kv.D == 128 ? launch_tile<__nv_bfloat16, 128>(a, st)
                             : launch_tile<__nv_bfloat16, 256>(a, st);
  }
}

}  // namespace np
