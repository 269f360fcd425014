// Shared by the kernels of attention over a paged cache: the problem, and how its work is cut.
//
// An item is a tile of BM rows (a row: a token and one of the G query heads that share a key head)
// of one request and key head. Its cost is what it takes to begin and end it and its tiles of KT keys,
// in units of about 0.3 us. The costs of all items in order are cut into equal shares, one per CTA, so
// that a long context is spread over many CTAs and a batch of ragged ones ends evenly; contexts are
// known on the device only, so every CTA adds up the requests' costs by itself and finds the start of
// its share. A share covers whole items and at most two cut ones (its first and its last piece). Pieces
// of cut items leave their rows' bases, sums and unnormalised outputs in the workspace, and the join
// kernel joins them in order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fast_div.cuh"
#include "gdp_internal.cuh"

namespace gdp {
namespace attn {

struct Problem {
  const void* q;
  int64_t qs[3];                  // batch, token, head
  const void *k, *v;              // caches
  int64_t ks[3], vs[3];           // page, token, head
  int n_pages, block;
  const int32_t* tables;          // [n, width]
  int width;
  const int32_t* ctx;             // [n]
  const int32_t* cu;              // null: n == B requests of T tokens
  int n, B, T, H, HKV, G, D, DV;
  Div by_G, by_block;
  const int64_t* tree;            // [B, T] or null: a chain
  float c;                        // scale log2 e
  gdp_dtype dt;
  void* o;                        // [B, T, H, DV]
  int32_t* status;                // may be null
  cudaStream_t stream;
};

// A cut item's record, in the entry of the CTA where it begins.
struct Rec {
  long long first;                // the request's first row of tokens in [B T]
  int row0, rows, head, more;     // rows == 0: none; more: CTAs after this one that hold pieces
};

// The begin and end of an item and a tile of keys, for items of up to 128 rows and for larger ones.
struct Cost {
  int begin, tile, begin2, tile2;
};

struct Args {
  Problem p;
  Cost cost;
  Rec* recs;                      // [ctas]
  float* part;                    // [ctas][2][dvp / 4][cap][4] outputs
  float2* ml;                     // [ctas][2][cap] base (log2) that the row's weights are relative to, and their sum
  int ctas, cap, dvp;             // cap: rows of a piece that are kept
};

struct Layout {
  size_t recs, ml, part, total;
  int cap, dvp;
};
inline Layout layout(int ctas, int64_t rows, int bm, int DV) {
  Layout x;
  x.cap = (int)(rows < bm ? rows : bm);
  x.dvp = (DV + 3) / 4 * 4;
  x.recs = 0;
  x.ml = align_up(sizeof(Rec) * (size_t)ctas);
  x.part = align_up(x.ml + sizeof(float2) * 2 * (size_t)ctas * x.cap);
  x.total = align_up(x.part + sizeof(float) * 2 * (size_t)ctas * x.cap * x.dvp);
  return x;
}

// What the rows of one request are. A request that is not `live` sees nothing (its rows are 0): padding, whose
// last new token has no page, or `bad` lengths.
struct Req {
  int S, ctx;
  bool live, bad;
};
__device__ __forceinline__ Req request(const Problem& p, int r) {
  Req x;
  x.S = p.cu ? p.cu[r + 1] - p.cu[r] : p.T;
  x.ctx = p.ctx[r];
  x.bad = x.ctx < 0 || (int64_t)x.ctx + x.S > (int64_t)p.width * p.block || (p.tree && x.S > 64);
  x.live = !x.bad && x.S > 0 &&
           p.tables[(int64_t)r * p.width + quot(x.ctx + x.S - 1, p.by_block)] >= 0;
  return x;
}
__device__ __forceinline__ int64_t first_row(const Problem& p, int r) {
  return p.cu ? p.cu[r] : (int64_t)r * p.T;
}

// (Rows of a request, S G, stay below 2^31 - 1024.)
template <int BM, int KT>
struct Cut {
  __device__ static __forceinline__ int tiles(const Problem& p, int S) { return (S * p.G + BM - 1) / BM; }
  // keys that the rows of a tile see at most
  __device__ static __forceinline__ int keys(const Problem& p, const Req& x, int tile) {
    if (!x.live) return 0;
    if (p.tree) return x.ctx + x.S;
    const int last = min((tile + 1) * BM, x.S * p.G) - 1;
    return x.ctx + (int)quot(last, p.by_G) + 1;
  }
  __device__ static __forceinline__ int units(int keys) { return keys > 0 ? (keys + KT - 1) / KT : 1; }
  __device__ static __forceinline__ bool large(const Problem& p, const Req& x, int tile) {
    return BM > 128 && x.S * p.G - tile * BM > 128;
  }
  __device__ static __forceinline__ int begin(const Cost& c, bool large) { return large ? c.begin2 : c.begin; }
  __device__ static __forceinline__ int each(const Cost& c, bool large) { return large ? c.tile2 : c.tile; }
  // (fits 32 bits: keys do, and a tile of 32 of them costs at most 8)
  __device__ static __forceinline__ int cost(const Problem& p, const Cost& c, const Req& x, int tile) {
    const bool l = large(p, x, tile);
    return begin(c, l) + units(keys(p, x, tile)) * each(c, l);
  }
  // of one head of a request
  __device__ static __forceinline__ int64_t head_cost(const Problem& p, const Cost& c, const Req& x) {
    if (x.S <= 0) return 0;
    const int n = tiles(p, x.S);
    if (p.tree || !x.live) return (int64_t)(n - 1) * cost(p, c, x, 0) + cost(p, c, x, n - 1);
    int64_t u = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) u += cost(p, c, x, i);
    return u;
  }
  // tiles of an item's keys that lie before a cut `at` units behind its begin
  __device__ static __forceinline__ int before(const Cost& c, bool large, long long at, int units) {
    const int each_ = each(c, large);
    at -= begin(c, large);
    return at <= 0 ? 0 : at >= (long long)units * each_ ? units : ((int)at + each_ - 1) / each_;
  }
};

// Where a CTA's share begins: an item, and how far in it; its length in units.
struct Start {
  int r, head, tile, bad;
  long long in, left, total, ctas, at;  // at: the share's first unit
};

// (32 bits where they do: the 64-bit division is a call of a hundred instructions.)
__device__ __forceinline__ long long divide(long long a, long long b) {
  return (a | b) >> 31 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// By all NT threads of the CTA. (64-bit sums: requests times heads times tiles may pass 2^31.)
template <int BM, int KT, int NT>
__device__ __forceinline__ void find_start(const Args& a, Start* out, long long* scratch /* [NT / 32 + 1] */) {
  const Problem& p = a.p;
  using C = Cut<BM, KT>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.n + NT - 1) / NT;
  const int r0 = (int)min((int64_t)tid * per, (int64_t)p.n), r1 = min(r0 + per, p.n);
  long long mine = 0, head = 0;  // head: of one head of the last request
  int bad = 0, odd = 0;
  Req x{};
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    if (p.cu) {
      const int a0 = p.cu[r], a1 = p.cu[r + 1];
      if (a0 < 0 || a1 < a0 || a1 > p.T || (r == 0 && a0 != 0)) { bad = 1; break; }
    }
    x = request(p, r);
    if (x.bad) odd = 1;
    head = C::head_cost(p, a.cost, x);
    mine += head;
  }
  mine *= p.HKV;
  if (blockIdx.x == 0 && (odd || bad)) report(p.status, GDP_ERR_INVALID_ARG);
  bad = __syncthreads_or(bad);
  long long sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) scratch[warp] = sum;
  if (tid == 0) { out->bad = bad; out->left = 0; }
  __syncthreads();
  long long before = sum - mine, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  // (no share is shorter than a tile, so that every CTA between a cut item's first and last has a piece)
  const long long ctas = max(1ll, min((long long)a.ctas, total / max(a.cost.tile, a.cost.tile2)));
  if (tid == 0) { out->total = total; out->ctas = ctas; }
  if (!bad && total > 0 && blockIdx.x < ctas) {
    // first unit of CTA c: floor(total c / ctas)
    const long long q = divide(total, ctas), rest = total - q * ctas;
    const long long u0 = q * blockIdx.x + divide(rest * blockIdx.x, ctas);
    if (before <= u0 && u0 < before + mine) {  // the thread whose requests hold the start
      long long at = u0 - before;
      int r = r0;
      if (r1 - r0 > 1)
#pragma unroll 1
        for (;; ++r) {
          x = request(p, r);
          head = C::head_cost(p, a.cost, x);
          if (at < head * p.HKV) break;
          at -= head * p.HKV;
        }
      const long long h = divide(at, head);
      at -= h * head;
      int tile = 0;
#pragma unroll 1
      for (;; ++tile) {
        const int u = C::cost(p, a.cost, x, tile);
        if (at < u) break;
        at -= u;
      }
      out->r = r;
      out->head = (int)h;
      out->tile = tile;
      out->in = at;
      out->left = q * (blockIdx.x + 1ll) + divide(rest * (blockIdx.x + 1ll), ctas) - u0;
      out->at = u0;
    }
  }
  __syncthreads();
}

// First unit of CTA c's share is floor(total c / ctas), so the last CTA with a unit before `end` is
// ceil(end ctas / total) - 1.
__device__ __forceinline__ int last_cta(long long end, long long ctas, long long total) {
  return (int)divide(end * ctas + total - 1, total) - 1;
}

// One piece of an item, and the walk over the pieces of a share.
struct Piece {
  Req x;
  int64_t first;       // the request's first row in [B T]
  int r, head, tile;
  int row0, rows;      // rows of the request's S G that the tile holds
  int keys;            // that the tile sees
  int j0, j1, units;   // key tiles of this piece, of the item
  int slot;            // of the partial results; -1: the item is whole
  long long end;       // the unit behind the first one of the item's last tile
};

template <int BM, int KT>
struct Walk {
  using C = Cut<BM, KT>;
  Cost cost;
  int r, head, tile;
  long long in, left, at;  // at: the item's first unit
  __device__ __forceinline__ Walk(const Start& s, const Cost& c)
      : cost(c), r(s.r), head(s.head), tile(s.tile), in(s.in), left(s.left), at(s.at - s.in) {}
  __device__ __forceinline__ bool next(const Problem& p, Piece& x) {
#pragma unroll 1
    while (left > 0) {
      x.x = request(p, r);
      while (x.x.S <= 0) x.x = request(p, ++r);  // (units are left, so there is one)
      x.first = first_row(p, r);
      x.r = r;
      x.head = head;
      x.tile = tile;
      x.row0 = tile * BM;
      x.rows = min(BM, x.x.S * p.G - x.row0);
      x.keys = C::keys(p, x.x, tile);
      x.units = C::units(x.keys);
      const bool large = C::large(p, x.x, tile);
      const long long all = C::begin(cost, large) + (long long)x.units * C::each(cost, large);
      x.j0 = C::before(cost, large, in, x.units);
      x.j1 = C::before(cost, large, in + left, x.units);
      x.slot = x.j0 == 0 && x.j1 == x.units ? -1 : x.j0 == 0 ? 1 : 0;
      // the unit in which the last tile begins, for the record of a cut item
      x.end = at + all - C::each(cost, large) + 1;
      left -= all - in;
      at += all;
      in = 0;
      if (++tile == C::tiles(p, x.x.S)) {
        tile = 0;
        if (++head == p.HKV) { head = 0; ++r; }
      }
      if (x.j1 > x.j0) return true;
    }
    return false;
  }
};

// Row R of a request: token R / G, query head head G + R % G.
__device__ __forceinline__ int64_t out_at(const Problem& p, int64_t first, int head, int row) {
  const int t = (int)quot(row, p.by_G);
  return ((first + t) * p.H + head * p.G + (row - t * p.G)) * (int64_t)p.DV;
}

// The record of a CTA's share: the piece that begins an item which goes on elsewhere, if there is one.
__device__ __forceinline__ void write_rec(const Args& a, const Start& s, const Piece* x) {
  Rec& r = a.recs[blockIdx.x];
  if (!x) {
    r.rows = 0;
    return;
  }
  r.first = x->first;
  r.row0 = x->row0;
  r.rows = x->rows;
  r.head = x->head;
  r.more = last_cta(x->end, s.ctas, s.total) - (int)blockIdx.x;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

void set_layout(Args& a, const Layout& x, uint8_t* ws, int ctas);

// The kernel for any type and size, and the one on the tensor cores: whether sizes and type fit it,
// whether addresses and strides do too (for TMA). Workspaces for requests of up to `rows` rows.
cudaError_t launch_simple(const Problem& p, uint8_t* ws);
size_t simple_workspace(int64_t rows, int DV);
bool tc_shape(int D, int DV, gdp_dtype dt);
bool tc_ok(const Problem& p);
size_t tc_workspace(int64_t rows, int D, int DV);
cudaError_t launch_tc(const Problem& p, uint8_t* ws);
// Test hook (gdp_debug_wait_fault): a wait of its next launch runs out (arm), limit of its waits.
void wait_fault(int arm, unsigned long long budget_ns);
cudaError_t launch_combine(const Args& a);

}  // namespace attn
}  // namespace gdp
