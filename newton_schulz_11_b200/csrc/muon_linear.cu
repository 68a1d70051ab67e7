// Linear layers and their gradients: the C ABI entry points, the plan of each product, and
// the elementwise kernels.
//
//   muon_linear               z = x W^T + bias,  y = act(z) + residual
//   muon_linear_backward      dx = (dy W) act'(z_in) + skip,  dW (+)= dy^T x,  db (+)= sum of dy
//   muon_activation_backward  dz = dy act'(z)
//
// Workspace: the operands that the tensor cores cannot read in place (fp32 ones, as bf16
// terms; bf16 ones whose rows are not 16-byte aligned, copied), the partial sums of split
// reductions, and those of the bias gradient, behind the step's header (kHeaderBytes).  Nothing
// in it outlives the call.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "muon_epilogue.cuh"
#include "muon_layers_host.h"

namespace muon {

struct ActGradParams {
  EpiView dy, z, dz;
  Sweep sweep;
  int32_t cols, act, wide;
};

// Eight columns of a row per thread and step; in whole rows of 16-column groups (p.wide) 16,
// 32 bytes of each bf16 operand at a time.  HBM-bound, with the instructions of the derivative
// close behind: 16384 x 4096 bf16 GELU (tanh) in 64.7 us, 97% of the measured copy bandwidth
// (84.8 us eight columns at a time).
__global__ void __launch_bounds__(256, 5) muon_activation_backward_kernel(const __grid_constant__ ActGradParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const Sweep& s = p.sweep;
  const int along = 1 << s.shift, deep = 256 >> s.shift;
  const int rb = blockIdx.x / s.col_blocks, cb = blockIdx.x - rb * s.col_blocks;
  const int g0 = (cb << s.shift) + (threadIdx.x & (along - 1));
  for (int64_t r = static_cast<int64_t>(rb) * deep + (threadIdx.x >> s.shift); r < s.rows;
       r += static_cast<int64_t>(s.row_blocks) * deep)
    for (int gr = g0; gr < s.groups; gr += s.col_blocks << s.shift) {
      if (p.wide) {
        const int c = gr * 16;
        const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(p.dy.p) + r * p.dy.ld + c;
        const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(p.z.p) + r * p.z.ld + c;
        uint4 a, b, e, f;
        ld_global_v8(dy, a, b);
        ld_global_v8(z, e, f);
        const uint32_t gw[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const uint32_t zw[8] = {e.x, e.y, e.z, e.w, f.x, f.y, f.z, f.w};
        F2 g[8], t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g[j] = EpiRow<16>::value(gw[j]);
          t[j] = EpiRow<16>::value(zw[j]);
        }
        apply_slope<8>(p.act, t, g);
        EpiRow<16>::store(reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(p.dz.p) + r * p.dz.ld + c), g);
      } else {
        const int c = gr * 8, valid = p.cols - c;
        F2 g[4], z[4];
        load_pairs<8>(p.dy, r * p.dy.ld + c, valid, g);
        load_pairs<8>(p.z, r * p.z.ld + c, valid, z);
        apply_slope<4>(p.act, z, g);
        store_pairs<8>(p.dz, r * p.dz.ld + c, valid, g);
      }
    }
}

}  // namespace muon

namespace {
using namespace muon;

// The plan counts the SMs of the one part this library is built for, so that a workspace
// can be sized without a device.
constexpr int kSms = 148;
constexpr int64_t kFlipTokens = 64;  // most tokens the flipped tiles take

bool sizes_ok(int64_t rows, int64_t in, int64_t out) {
  return rows >= 0 && rows <= kMaxRows && in >= 1 && in <= kMaxSide && out >= 1 && out <= kMaxSide;
}

bool act_ok(int act) { return act >= MUON_ACT_NONE && act <= MUON_ACT_SILU; }

// k-blocks per piece of a Sum variant: 512 of k for bf16 operands, 256 where a k-block is
// several term products, which hide the reading of the accumulator as well.  (fp32 products
// 512 at a time are off by 5e-7 relative and 1% quicker; 256 by 2.8e-7; 128 by 1.8e-7, 3 to 5%
// slower.)  A bf16 result does not show that much: its large products take 2048 at a time,
// off by 2.3e-6, which cost 1% of 4096 x 16384 x 4096 (431 and 435 us).
int64_t piece_blocks(int nseg, bool pair, bool bf16_out) { return pair && bf16_out ? 32 : nseg == 1 ? 8 : 4; }

// The longest reduction of a bf16 result that stays in the accumulator as a whole: there the
// truncation has grown to 4.5e-6 relative for zero-mean products, 1.3e-5 for products of one
// sign (a 300th of the result's half step, 2^-8), and pieces of 2048 would cost
// 8192 x 4096 x 14336 2% and 8192 x 4096 x 1024 with a residual 8%.
constexpr int64_t kWholeReduction = 4096;

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// An operand of a product: a stored matrix as the tensor cores will read it.
struct Operand {
  const muon_view_t* v = nullptr;
  int64_t rows = 0, cols = 0;
  int terms = 1;
  bool direct = true;     // read in place
  size_t offset = 0;      // of the packed terms in the workspace
  int64_t ld_packed = 0;  // elements, a multiple of 8

  Operand() = default;
  Operand(const muon_view_t& view, int64_t r, int64_t c) : v(&view), rows(r), cols(c) {
    terms = view.dtype == MUON_F32 ? kTerms : 1;
    const int64_t ld = row_stride(view, r, c);
    direct = terms == 1 && aligned_bytes(view.data, 16) && (r <= 1 || ld % 8 == 0);
    ld_packed = ceil_div(c, 8) * 8;
  }
  size_t term_bytes() const { return up(static_cast<size_t>(rows) * ld_packed * 2); }
  size_t bytes() const { return direct ? 0 : terms * term_bytes(); }
  void place(size_t* at) {
    offset = *at;
    *at += bytes();
  }
};

// How a product runs.  m, n: the output's rows and columns; k: the reduction.
struct Plan {
  int tile = kOne128;
  int64_t tiles_m = 0, tiles_n = 0, nk = 0, splits = 1, kb_per_split = 0;
  int nseg = 1;
  bool shared = false;  // launched with the call's other product
  size_t partial_bytes = 0;
  int64_t ld_partial = 0;
  double cost = 0.0;
};

int segments(int ta, int tb) { return ta == 1 ? tb : (tb == 1 ? ta : kMaxSegments); }

// What a plan depends on besides the sizes.
struct PlanTraits {
  int nseg;      // term products
  bool sum;      // the reduction is added in pieces
  bool tokens;   // the output's rows are tokens
  bool aligned;  // the epilogue's rows can be accessed 16 bytes at a time
};

// The estimated time of a product in SM cycles, fitted to measurements (captured calls, us):
//   a k-block of 64 takes a CTA or a pair about 0.4 us of 128 x 128 or 256 x 256 alike, since
//   both wait for 32 KB a CTA: 1024 x 1024 x 8192 in 64 single tiles 54, in 16 pair tiles 55;
//   a split of a large product costs about 3 us and its traffic: 1024 x 1024 x 8192 takes 55,
//   35, 24.7, 30.8 in 1, 2, 4 and 8 splits; 2048 x 1024 x 1024 takes 11.0, and 15.3 in 2.
double pair_cost(const TileShape& shape, int64_t tiles, int64_t splits, int64_t per, int64_t outputs, int nseg) {
  double start = shape.sum ? 2200.0 : 1500.0;
  if (shape.flip) start += 5000.0;  // 128 outputs a thread, one by one
  const double waves = static_cast<double>(ceil_div(tiles * splits, kSms / 2));
  const double cost = waves * (static_cast<double>(per) * 760.0 * nseg + start);
  return splits == 1 ? cost : cost + 5500.0 + static_cast<double>((splits + 1) * outputs) * 4.0 / 2600.0;
}

// Clusters of small products that run at the same time (what the occupancy calculator says).
int64_t clusters_at_once(int64_t size) { return size == 1 ? kSms : size == 2 ? 74 : size == 4 ? 33 : 15; }

//   a small product loads each term of a k-block once; it has its launch's start, its epilogue,
//   which the cluster divides, and the cluster's two barriers
double small_cost(const TileShape& shape, int64_t tiles, int64_t cluster, int64_t nk, int nseg) {
  const double waves = static_cast<double>(ceil_div(tiles, clusters_at_once(cluster)));
  const double block = shape.n == 128 ? 760.0 : 700.0;
  const double loads = nseg == 1 ? 1.0 : nseg == kTerms ? 2.0 : 3.0;  // of a bf16 product's
  return waves * (static_cast<double>(ceil_div(nk, cluster)) * block * loads + 2500.0 + 30.0 * shape.n / cluster) +
         (cluster > 1 ? 2500.0 : 0.0);
}

// Picks the tile and the number of splits with the least estimated time.
Plan search_plan(int64_t m, int64_t n, int64_t k, const PlanTraits& t) {
  Plan best;
  best.cost = 1e30;
  best.nk = ceil_div(k, kProductBK);
  best.nseg = t.nseg;
  const bool few = t.tokens && m <= kFlipTokens;
  for (int tile = kPair256; tile <= kFlip64; ++tile) {
    const TileShape& shape = kTileShapes[tile];
    if (shape.pair && (shape.sum != t.sum || few)) continue;
    if (tile >= kFlip32 ? !few || m > shape.n : few) continue;
    const int64_t tm = ceil_div(shape.flip ? n : m, shape.m), tn = ceil_div(shape.flip ? m : n, shape.n);
    for (int64_t want = 1; want <= (shape.pair ? 32 : 8); shape.pair ? ++want : want *= 2) {
      const int64_t per = ceil_div(best.nk, want);
      if (tm * tn * want > 0x3fffffff) break;
      // (partial sums are aligned whatever the output is)
      const bool flip = !t.aligned && (!shape.pair || want == 1);
      if (!few && shape.flip != flip) continue;
      if (shape.pair && (ceil_div(best.nk, per) != want || (want > 1 && per < 2))) continue;
      const double cost = shape.pair ? pair_cost(shape, tm * tn, want, per, m * n, t.nseg)
                                     : small_cost(shape, tm * tn, want, best.nk, t.nseg);
      if (cost < best.cost) {
        best.cost = cost;
        best.tile = tile;
        best.tiles_m = tm;
        best.tiles_n = tn;
        best.splits = want;
        best.kb_per_split = per;
      }
    }
  }
  if (kTileShapes[best.tile].pair && best.splits > 1) {
    best.ld_partial = ceil_div(n, 32) * 32;
    best.partial_bytes = up(static_cast<size_t>(best.splits) * m * best.ld_partial * 4);
  }
  return best;
}

// Two products of a call as small ones in one launch, where that beats one after the other
// (their times and a launch of about 3000 cycles between them).
void share_launch(Plan* a, int64_t am, int64_t an, Plan* b, int64_t bm, int64_t bn, bool aligned) {
  const int tile = aligned ? kOne128 : kFlip128;
  const TileShape& shape = kTileShapes[tile];
  const int64_t atm = ceil_div(aligned ? am : an, 128), atn = ceil_div(aligned ? an : am, 128);
  const int64_t btm = ceil_div(aligned ? bm : bn, 128), btn = ceil_div(aligned ? bn : bm, 128);
  double least = a->cost + b->cost + 3000.0;
  for (int64_t ca = 1; ca <= 8; ca *= 2)
    for (int64_t cb = 1; cb <= 8; cb *= 2) {  // a cluster holds several tiles of the product that is split less
      const int64_t c = std::max(ca, cb);
      if (ceil_div(atm * atn * ca, c) + ceil_div(btm * btn * cb, c) > clusters_at_once(c)) continue;
      const double cost = std::max(small_cost(shape, atm * atn, ca, a->nk, a->nseg),
                                   small_cost(shape, btm * btn, cb, b->nk, b->nseg));
      if (cost >= least) continue;
      least = cost;
      a->shared = b->shared = true;
      a->tile = b->tile = tile;
      a->splits = ca;
      b->splits = cb;
      a->tiles_m = atm;
      a->tiles_n = atn;
      b->tiles_m = btm;
      b->tiles_n = btn;
      a->partial_bytes = b->partial_bytes = 0;
    }
}

// The search takes a microsecond or two; a call asks for its plan twice (its workspace, then
// itself), and a training loop for the same few sizes again and again.
Plan make_plan(int64_t m, int64_t n, int64_t k, const PlanTraits& t) {
  struct Entry {
    int64_t m = -1, n = 0, k = 0;
    int flags = 0;
    Plan plan;
  };
  static thread_local Entry table[64];
  const int flags = t.nseg * 8 + (t.sum ? 4 : 0) + (t.tokens ? 2 : 0) + (t.aligned ? 1 : 0);
  uint64_t h = static_cast<uint64_t>(m) * 0x9E3779B97F4A7C15ull;
  h = (h ^ static_cast<uint64_t>(n)) * 0x9E3779B97F4A7C15ull;
  h = (h ^ static_cast<uint64_t>(k)) * 0x9E3779B97F4A7C15ull;
  Entry& e = table[((h >> 32) ^ static_cast<uint64_t>(flags)) % 64];
  if (e.m != m || e.n != n || e.k != k || e.flags != flags) {
    e.plan = search_plan(m, n, k, t);
    e.m = m;
    e.n = n;
    e.k = k;
    e.flags = flags;
  }
  return e.plan;
}

// Adds the layout of `o` to the call's first launch, unless it is read in place.
void add_pack(PrepareParams* p, const Operand& o, uint8_t* ws) {
  if (o.direct || o.rows == 0) return;
  PackTask& t = p->pack[p->packs];
  t.src = epi_view(*o.v, o.rows, o.cols);
  t.dst = reinterpret_cast<__nv_bfloat16*>(ws + o.offset);
  t.ld_dst = o.ld_packed;
  t.term_stride = static_cast<int64_t>(o.term_bytes() / 2);
  t.cols = static_cast<int32_t>(o.cols);
  t.terms = o.terms;
  t.sweep = make_sweep(ceil_div(o.rows, 2), o.ld_packed / 8, 8 * kSms);  // two rows a thread
  t.sweep.rows = o.rows;
  p->begin[p->packs + 1] = p->begin[p->packs] + sweep_blocks(t.sweep);
  ++p->packs;
}

// `side_rows`: how many of the operand's side a box of a K-major operand covers.
bool operand_maps(CUtensorMap* maps, const Operand& o, uint8_t* ws, bool mn, int side_rows) {
  for (int t = 0; t < o.terms; ++t) {
    const void* base = o.direct ? o.v->data : ws + o.offset + t * o.term_bytes();
    const int64_t ld = o.direct ? (o.rows <= 1 ? ceil_div(o.cols, 8) * 8 : o.v->ld) : o.ld_packed;
    if (!encode_operand_map(&maps[t], base, o.rows, o.cols, ld, mn ? 64 : side_rows)) return false;
  }
  return true;
}

bool plain_epilogue(const Epilogue& e) {
  for (const EpiView* v : {&e.preact, &e.slope, &e.add, &e.out})
    if (v->p != nullptr && !(v->bf16 && v->vec == 2)) return false;
  return e.bias.p == nullptr || e.bias.vec == 2;
}

// a: the operand on the output's row side; b: on its column side.  mn: contiguous along the
// side.  A split large product leaves its end to `finish`.
muon_status_t make_product(const Plan& pl, const Operand& a, bool a_mn, const Operand& b, bool b_mn, const Epilogue& e,
                           uint8_t* ws, size_t partial_at, FinishParams* finish, ProductParams* out) {
  static const uint8_t both_a[kMaxSegments] = {0, 2, 1, 0, 1, 0}, both_b[kMaxSegments] = {2, 0, 1, 1, 0, 0};
  const TileShape& shape = kTileShapes[pl.tile];
  const bool flip = shape.flip;
  const Operand &am = flip ? b : a, &bm = flip ? a : b;
  *out = ProductParams{};
  ProductParams& p = *out;
  p.a_mn = flip ? b_mn : a_mn;
  p.b_mn = flip ? a_mn : b_mn;
  if (!operand_maps(p.map_a, am, ws, p.a_mn, 128) ||
      !operand_maps(p.map_b, bm, ws, p.b_mn, shape.pair ? 128 : shape.n))
    return MUON_ERR_CUDA;
  p.e = e;
  p.e.plain = plain_epilogue(e);
  p.tiles_m = static_cast<int32_t>(pl.tiles_m);
  p.tiles_n = static_cast<int32_t>(pl.tiles_n);
  p.nk = static_cast<int32_t>(pl.nk);
  p.splits = static_cast<int32_t>(pl.splits);
  p.kb_per_split = static_cast<int32_t>(pl.kb_per_split);
  const bool bf16_out = e.out.bf16 && (e.preact.p == nullptr || e.preact.bf16);
  p.piece = shape.sum ? static_cast<int32_t>(piece_blocks(pl.nseg, shape.pair, bf16_out)) : p.kb_per_split;
  p.nseg = pl.nseg;
  p.walk = am.terms == 1 ? (bm.terms == 1 ? kWalkOne : kWalkCols) : (bm.terms == 1 ? kWalkRows : kWalkBoth);
  for (int g = 0; g < pl.nseg; ++g) {  // the smallest products first
    p.seg_a[g] = static_cast<uint8_t>(am.terms == 1 ? 0 : bm.terms == 1 ? pl.nseg - 1 - g : both_a[g]);
    p.seg_b[g] = static_cast<uint8_t>(bm.terms == 1 ? 0 : am.terms == 1 ? pl.nseg - 1 - g : both_b[g]);
  }
  p.timeout_ns = layers_wait_ns();
  if (shape.pair && pl.splits > 1) {
    p.partial = reinterpret_cast<float*>(ws + partial_at);
    p.ld_partial = pl.ld_partial;
    p.split_stride = e.rows * pl.ld_partial;
    JoinTask& j = finish->join[finish->joins];
    j.e = e;
    j.partial = p.partial;
    j.ld_partial = p.ld_partial;
    j.split_stride = p.split_stride;
    j.splits = p.splits;
    j.sweep = make_sweep(e.rows, ceil_div(e.cols, 8), 8 * kSms);
    finish->begin[finish->joins + 1] = finish->begin[finish->joins] + sweep_blocks(j.sweep);
    ++finish->joins;
  }
  return MUON_OK;
}

// Blocks of a small product in clusters of `cluster`.
int small_blocks(const Plan& pl, int64_t cluster) {
  return static_cast<int>(ceil_div(pl.tiles_m * pl.tiles_n * pl.splits, cluster) * cluster);
}

// Launches p (already made), or two small products that share a launch.
muon_status_t run_product(const Plan& pl, ProductGroup& g, const Plan* second, cudaStream_t s) {
  if (kTileShapes[pl.tile].pair) return queued(launch_product_pair(pl.tile, g.p[0], kSms, s));
  g.cluster = static_cast<int32_t>(second == nullptr ? pl.splits : std::max(pl.splits, second->splits));
  g.first_blocks = small_blocks(pl, g.cluster);
  const int blocks = g.first_blocks + (second == nullptr ? 0 : small_blocks(*second, g.cluster));
  return queued(launch_product_small(pl.tile, g, blocks, s));
}

// Whether the rows of an epilogue operand (if it is there) can be accessed 16 bytes at a time.
bool wide_rows(const muon_view_t& v, int64_t rows, int64_t cols) {
  return v.data == nullptr || epi_view(v, rows, cols).vec > 0;
}

bool wants_sum(const muon_view_t& out, int64_t k) {
  return out.data != nullptr && (out.dtype == MUON_F32 || k > kWholeReduction);
}

struct LinearPlan {
  Operand x, w;
  Plan z;
  size_t partial_at = 0, bytes = 0;  // from the start of the workspace, whose header is left alone
};

LinearPlan plan_linear(const muon_linear_t* d) {
  LinearPlan pl;
  if (d->rows == 0) return pl;
  pl.bytes = kHeaderBytes;
  pl.x = Operand(d->x, d->rows, d->in);
  pl.w = Operand(d->w, d->out, d->in);
  const bool aligned = wide_rows(d->y, d->rows, d->out) && wide_rows(d->preact, d->rows, d->out) &&
                       wide_rows(d->residual, d->rows, d->out);
  pl.z = make_plan(d->rows, d->out, d->in, {segments(pl.x.terms, pl.w.terms),
                                            wants_sum(d->y, d->in) || wants_sum(d->preact, d->in), true,
                                            aligned});
  pl.x.place(&pl.bytes);
  pl.w.place(&pl.bytes);
  pl.partial_at = pl.bytes;
  pl.bytes += pl.z.partial_bytes;
  if (pl.bytes == kHeaderBytes) pl.bytes = 0;
  return pl;
}

struct LinearGradPlan {
  Operand dy, x, w;
  Plan dx, dw;
  int64_t slices = 0;
  int sum_blocks = 0;  // of the last product's launch that sum columns; 0: in the first launch
  size_t dx_at = 0, dw_at = 0, db_at = 0, bytes = 0;
};

// How many blocks that would be idle under the call's last product can sum the columns of dy
// in less time than that product takes, or 0.  A block takes 256 rows of 64 columns in about
// a microsecond, a product 0.4 us a k-block.  Measured, with the sums riding and with them in
// the first launch (us): 515 x 770 x 1030 fp32 33.8, 39.0; 1000 x 1000 x 1000 bf16 18, 21.8;
// 8192 x 4096 x 1024 bf16 132 to 135, 140.
int idle_blocks(const Plan& last, const Plan& other, int64_t tasks, int64_t rows) {
  const bool pair = kTileShapes[last.tile].pair;
  const int size = pair ? 2 : static_cast<int>(last.shared ? std::max(last.splits, other.splits) : last.splits);
  int64_t used = pair ? 2 * last.tiles_m * last.tiles_n * last.splits : small_blocks(last, size);
  if (last.shared) used += small_blocks(other, size);
  int64_t idle = (kSms - used) / size * size;
  if (size > 2) idle = std::min<int64_t>(idle, clusters_at_once(size) * size - used);
  idle = std::min(idle, ceil_div(tasks, size) * size);
  if (idle <= 0) return 0;
  const double sums = static_cast<double>(ceil_div(tasks, idle)) * (static_cast<double>(rows) / 256.0 + 2.0);
  const double product =
      4.0 + 0.4 * (pair ? last.nseg * last.kb_per_split : (last.nseg + 1) / 2 * ceil_div(last.nk, last.splits));
  return sums <= product ? static_cast<int>(idle) : 0;
}

LinearGradPlan plan_linear_grad(const muon_linear_grad_t* d) {
  LinearGradPlan pl;
  if (d->rows == 0) return pl;
  const bool dx = d->dx.data != nullptr, dw = d->dw.data != nullptr;
  bool dx_aligned = true;
  pl.bytes = kHeaderBytes;
  pl.dy = Operand(d->dy, d->rows, d->out);
  if (dx || dw) pl.dy.place(&pl.bytes);
  if (dx) {
    pl.w = Operand(d->w, d->out, d->in);
    pl.w.place(&pl.bytes);
    dx_aligned = wide_rows(d->dx, d->rows, d->in) && wide_rows(d->skip, d->rows, d->in) &&
                 (d->in_act == MUON_ACT_NONE || wide_rows(d->preact, d->rows, d->in));
    pl.dx = make_plan(d->rows, d->in, d->out,
                      {segments(pl.dy.terms, pl.w.terms), wants_sum(d->dx, d->out), true, dx_aligned});
  }
  if (dw) {
    pl.x = Operand(d->x, d->rows, d->in);
    pl.x.place(&pl.bytes);
    pl.dw = make_plan(d->out, d->in, d->rows, {segments(pl.dy.terms, pl.x.terms), true, false,
                                               wide_rows(d->dw, d->out, d->in)});
    const bool same = wide_rows(d->dw, d->out, d->in) == dx_aligned;
    if (dx && same) share_launch(&pl.dx, d->rows, d->in, &pl.dw, d->out, d->in, dx_aligned);
    pl.dw_at = pl.bytes;
    pl.bytes += pl.dw.partial_bytes;
  }
  pl.dx_at = pl.bytes;
  pl.bytes += pl.dx.partial_bytes;
  if (d->db != nullptr) {
    const int64_t tasks = ceil_div(d->out, 64);
    pl.sum_blocks = dx || dw ? idle_blocks(dw ? pl.dw : pl.dx, pl.dx, tasks, d->rows) : 0;
    // a block's 256 threads cover 256 rows of 64 columns in one batch of loads (512 rows a
    // block: 7.9 us for 2000 x 2000 fp32 where 256 took 5.4; 7.6 and 6.4 for 8192 x 1024 bf16)
    pl.slices = pl.sum_blocks > 0 ? 1 : std::max<int64_t>(1, std::min(d->rows / 256, 8 * kSms / tasks));
    pl.db_at = pl.bytes;
    if (pl.slices > 1) pl.bytes += up(static_cast<size_t>(pl.slices) * d->out * 4);
  }
  if (pl.bytes == kHeaderBytes) pl.bytes = 0;
  return pl;
}

// Lets the last product's launch sum the columns, where the plan says so.
void add_sums(const LinearGradPlan& pl, int64_t cols, const ColumnSumTask& sum, ProductGroup* g) {
  if (pl.sum_blocks == 0) return;
  g->p[0].sum = sum;
  g->p[0].sum_tasks = static_cast<int32_t>(ceil_div(cols, 64));
  g->p[0].sum_blocks = pl.sum_blocks;
}

muon_status_t take_workspace(Operands* ops, void* ws, size_t have, size_t need) {
  if (ops->status != MUON_OK || need == 0) return ops->status;
  if (ws == nullptr || have < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned_bytes(ws, 256)) return MUON_ERR_ALIGNMENT;
  ops->add_bytes(ws, need);
  return MUON_OK;
}

// The checks of a descriptor without its workspace, so that sizing a call checks it too.
muon_status_t check_linear(const muon_linear_t* d, Operands* ops) {
  if (d == nullptr || !act_ok(d->act)) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->in, d->out)) return MUON_ERR_UNSUPPORTED_SHAPE;
  ops->add(d->x, d->rows, d->in, true, false);
  ops->add(d->w, d->out, d->in, true, false);
  ops->add(d->bias, 1, d->out, false, false);
  if (!same_view(d->y, d->residual, d->rows)) ops->add(d->residual, d->rows, d->out, false, false);
  ops->add(d->y, d->rows, d->out, true, true);
  ops->add(d->preact, d->rows, d->out, false, true);
  return ops->status;
}

muon_status_t check_linear_grad(const muon_linear_grad_t* d, Operands* ops) {
  if (d == nullptr || !act_ok(d->in_act) || (d->accumulate != 0 && d->accumulate != 1)) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->in, d->out)) return MUON_ERR_UNSUPPORTED_SHAPE;
  const bool dx = d->dx.data != nullptr, dw = d->dw.data != nullptr, slope = dx && d->in_act != MUON_ACT_NONE;
  ops->add(d->dy, d->rows, d->out, true, false);
  ops->add(d->x, d->rows, d->in, dw, false);
  ops->add(d->w, d->out, d->in, dx, false);
  ops->add(d->preact, d->rows, d->in, slope, false);
  if (!(dx && same_view(d->dx, d->skip, d->rows))) ops->add(d->skip, d->rows, d->in, false, false);
  ops->add(d->dx, d->rows, d->in, false, true);
  ops->add(d->dw, d->out, d->in, false, true);
  ops->add_f32(d->db, d->out, false, true);
  if (dw && d->dw.dtype != MUON_F32) ops->fail(MUON_ERR_UNSUPPORTED_DTYPE);
  if (!dx && !dw && d->db == nullptr && d->rows > 0) ops->fail(MUON_ERR_INVALID_ARG);
  return ops->status;
}

}  // namespace

extern "C" {

muon_status_t muon_linear_workspace(const muon_linear_t* d, size_t* bytes) {
  Operands ops;
  const muon_status_t st = check_linear(d, &ops);
  if (st != MUON_OK) return st;
  if (bytes == nullptr) return MUON_ERR_INVALID_ARG;
  *bytes = plan_linear(d).bytes;
  return MUON_OK;
}

muon_status_t muon_linear(const muon_linear_t* d, void* workspace, size_t workspace_bytes, void* stream) {
  Operands ops;
  muon_status_t st = check_linear(d, &ops);
  if (st != MUON_OK) return st;
  const LinearPlan pl = plan_linear(d);
  if ((st = take_workspace(&ops, workspace, workspace_bytes, pl.bytes)) != MUON_OK) return st;
  if ((st = ops.check()) != MUON_OK) return st;
  int sms = 0;
  if ((st = layers_device(&sms)) != MUON_OK) return st;
  if (d->rows == 0) return MUON_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PrepareParams before{};
  FinishParams after{};
  add_pack(&before, pl.x, ws);
  add_pack(&before, pl.w, ws);
  if (before.packs > 0) {
    before.begin[before.packs + 1] = before.begin[before.packs];
    if ((st = queued(launch_prepare(before, s))) != MUON_OK) return st;
  }
  Epilogue e{};
  e.rows = d->rows;
  e.cols = d->out;
  e.bias = epi_view(d->bias, 1, d->out);
  e.preact = epi_view(d->preact, d->rows, d->out);
  e.add = epi_view(d->residual, d->rows, d->out);
  e.out = epi_view(d->y, d->rows, d->out);
  e.act = d->act;
  ProductGroup g{};
  if ((st = make_product(pl.z, pl.x, false, pl.w, false, e, ws, pl.partial_at, &after, &g.p[0])) != MUON_OK) return st;
  st = run_product(pl.z, g, nullptr, s);
  if (st != MUON_OK || after.joins == 0) return st;
  after.begin[after.joins + 1] = after.begin[after.joins];
  return queued(launch_finish(after, s));
}

muon_status_t muon_linear_backward_workspace(const muon_linear_grad_t* d, size_t* bytes) {
  Operands ops;
  const muon_status_t st = check_linear_grad(d, &ops);
  if (st != MUON_OK) return st;
  if (bytes == nullptr) return MUON_ERR_INVALID_ARG;
  *bytes = plan_linear_grad(d).bytes;
  return MUON_OK;
}

muon_status_t muon_linear_backward(const muon_linear_grad_t* d, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  Operands ops;
  muon_status_t st = check_linear_grad(d, &ops);
  if (st != MUON_OK) return st;
  const LinearGradPlan pl = plan_linear_grad(d);
  if ((st = take_workspace(&ops, workspace, workspace_bytes, pl.bytes)) != MUON_OK) return st;
  if ((st = ops.check()) != MUON_OK) return st;
  int sms = 0;
  if ((st = layers_device(&sms)) != MUON_OK) return st;
  const bool dx = d->dx.data != nullptr, dw = d->dw.data != nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->rows == 0) {  // the sums are empty
    if (d->accumulate) return MUON_OK;
    const size_t pitch = static_cast<size_t>(row_stride(d->dw, d->out, d->in)) * 4;
    if (dw && cudaMemset2DAsync(d->dw.data, pitch, 0, static_cast<size_t>(d->in) * 4, d->out, s) != cudaSuccess)
      return MUON_ERR_CUDA;
    if (d->db != nullptr && cudaMemsetAsync(d->db, 0, static_cast<size_t>(d->out) * 4, s) != cudaSuccess)
      return MUON_ERR_CUDA;
    return MUON_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PrepareParams before{};
  FinishParams after{};
  if (dx || dw) add_pack(&before, pl.dy, ws);
  if (dx) add_pack(&before, pl.w, ws);
  if (dw) add_pack(&before, pl.x, ws);
  before.begin[before.packs + 1] = before.begin[before.packs];
  if (d->db != nullptr) {
    ColumnSumTask& t = before.sum;
    t.src = epi_view(d->dy, d->rows, d->out);
    t.out = d->db;
    t.partial = reinterpret_cast<float*>(ws + pl.db_at);
    t.rows = d->rows;
    t.cols = static_cast<int32_t>(d->out);
    t.accumulate = d->accumulate;
    t.slices = static_cast<int32_t>(pl.slices);
    if (pl.sum_blocks == 0) before.begin[before.packs + 1] += static_cast<int32_t>(ceil_div(d->out, 64) * pl.slices);
    after.sum = t;
  }
  if (before.begin[before.packs + 1] > 0)
    if ((st = queued(launch_prepare(before, s))) != MUON_OK) return st;
  ProductGroup g{};
  if (dx) {
    Epilogue e{};
    e.rows = d->rows;
    e.cols = d->in;
    if (d->in_act != MUON_ACT_NONE) {
      e.slope = epi_view(d->preact, d->rows, d->in);
      e.slope_act = d->in_act;
    }
    e.add = epi_view(d->skip, d->rows, d->in);
    e.out = epi_view(d->dx, d->rows, d->in);
    st = make_product(pl.dx, pl.dy, false, pl.w, true, e, ws, pl.dx_at, &after, &g.p[0]);
    if (!dw) add_sums(pl, d->out, after.sum, &g);
    if (st == MUON_OK && !pl.dx.shared) st = run_product(pl.dx, g, nullptr, s);
    if (st != MUON_OK) return st;
  }
  if (dw) {
    Epilogue e{};
    e.rows = d->out;
    e.cols = d->in;
    e.out = epi_view(d->dw, d->out, d->in);
    if (d->accumulate) e.add = e.out;
    const int at = pl.dw.shared ? 1 : 0;
    st = make_product(pl.dw, pl.dy, true, pl.x, true, e, ws, pl.dw_at, &after, &g.p[at]);
    add_sums(pl, d->out, after.sum, &g);
    if (st == MUON_OK) st = pl.dw.shared ? run_product(pl.dx, g, &pl.dw, s) : run_product(pl.dw, g, nullptr, s);
    if (st != MUON_OK) return st;
  }
  after.begin[after.joins + 1] = after.begin[after.joins];
  if (pl.slices > 1) after.begin[after.joins + 1] += static_cast<int32_t>(ceil_div(d->out, 32));
  return after.begin[after.joins + 1] > 0 ? queued(launch_finish(after, s)) : MUON_OK;
}

muon_status_t muon_activation_backward(const muon_activation_grad_t* d, void* stream) {
  if (d == nullptr || !act_ok(d->act) || d->act == MUON_ACT_NONE) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->cols, 1)) return MUON_ERR_UNSUPPORTED_SHAPE;
  Operands ops;
  ops.add(d->dy, d->rows, d->cols, true, false);
  ops.add(d->z, d->rows, d->cols, true, false);
  ops.add(d->dz, d->rows, d->cols, true, true);
  if (d->rows > 0 && d->dz.dtype != d->dy.dtype) ops.fail(MUON_ERR_UNSUPPORTED_DTYPE);
  muon_status_t st = ops.check();
  if (st != MUON_OK) return st;
  int sms = 0;
  if ((st = layers_device(&sms)) != MUON_OK) return st;
  if (d->rows == 0) return MUON_OK;
  ActGradParams p{};
  p.dy = epi_view(d->dy, d->rows, d->cols);
  p.z = epi_view(d->z, d->rows, d->cols);
  p.dz = epi_view(d->dz, d->rows, d->cols);
  p.wide = d->cols % 16 == 0;
  for (const EpiView* v : {&p.dy, &p.z, &p.dz})
    if (!v->bf16 || v->vec != 2) p.wide = 0;
  p.sweep = make_sweep(d->rows, ceil_div(d->cols, p.wide ? 16 : 8), 12 * kSms);
  p.cols = static_cast<int32_t>(d->cols);
  p.act = d->act;
  return queued(launch_dependent(muon_activation_backward_kernel, p,
                                 dim3(static_cast<unsigned>(sweep_blocks(p.sweep))), 256,
                                 static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
