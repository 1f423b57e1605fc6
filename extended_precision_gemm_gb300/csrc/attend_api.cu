// attend_api.cu -- the C entry points of rotary positions, the paged 4-bit cache and
// attention over it (declarations in ddgemm.h): argument checks, workspaces,
// launch sequences.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <numeric>

#include "attend.cuh"
#include "entry.cuh"

using namespace ddg;

namespace {

// A tokens x heads x dim array with its strides of tokens and heads.
struct Heads {
    const void* p;
    int64_t tokens, heads, dim, per_token, per_head, elem;

    // Heads and tokens that do not overlap, whichever of the two is the inner one,
    // within 2^62 bytes.
    bool sound() const {
        if (tokens == 0 || heads == 0 || dim == 0) return true;
        if (p == nullptr || (uintptr_t)p % elem != 0) return false;
        const long double t = tokens > 1 ? per_token : 0, h = heads > 1 ? per_head : 0;
        const long double all_tokens = (tokens - 1) * t, all_heads = (heads - 1) * h;
        if (t < 0 || h < 0 || (all_tokens + all_heads + dim) * elem > 4.6e18L) return false;
        if (heads > 1 && tokens > 1) return (h >= dim && t >= all_heads + dim) || (t >= dim && h >= all_tokens + dim);
        return (heads <= 1 || h >= dim) && (tokens <= 1 || t >= dim);
    }
    int64_t bytes() const {
        if (tokens == 0 || heads == 0 || dim == 0) return 0;
        return ((tokens - 1) * (tokens > 1 ? per_token : 0) + (heads - 1) * (heads > 1 ? per_head : 0) + dim) * elem;
    }
};
// Runs of `own` bytes from p on, every `period` bytes (0: one run) or at some of these places.
struct Runs {
    int64_t period, own;
};
// An array as runs of its heads' elements, or of what lies between two steps of its longer stride.
Runs runs_of(const Heads& a, bool longer) {
    const int64_t t = a.tokens > 1 ? a.per_token : 0, h = a.heads > 1 ? a.per_head : 0;
    if (!longer) return Runs{std::gcd(t, h) * a.elem, a.dim * a.elem};
    const bool token = t >= h;
    return Runs{(token ? t : h) * a.elem, ((token ? (a.heads - 1) * h : (a.tokens - 1) * t) + a.dim) * a.elem};
}
// Whether two arrays have an element in common, or could have: parts of one array side by side, heads of a token or
// halves of a head, have none although each reaches over the other.
bool meet(const Heads& a, const Heads& b) {
    if (!overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
    for (const bool la : {false, true}) {
        for (const bool lb : {false, true}) {
            const Runs x = runs_of(a, la), y = runs_of(b, lb);
            const int64_t period = std::gcd(x.period, y.period);
            if (period == 0) continue;
            int64_t from_x = ((int64_t)((uintptr_t)b.p - (uintptr_t)a.p)) % period;
            if (from_x < 0) from_x += period;
            if (x.own <= from_x && from_x + y.own <= period) return false;
        }
    }
    return true;
}

ddgemm_status check_cache(const ddgemm_mx4_cache* c, CacheView& v) {
    if (c == nullptr || !known_format(c->format) || c->pages < 0 || c->heads < 1 || c->head_dim < 1) return DDGEMM_ERR_INVALID_ARG;
    if (c->head_dim > 256 || c->heads > DDGEMM_MAX_HEADS || c->pages >= (1LL << 31)) return DDGEMM_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)) != 0) return DDGEMM_ERR_INVALID_ARG;
    if (c->pages > ((1LL << 34) - 1) / (c->page_size * c->heads)) return DDGEMM_ERR_UNSUPPORTED;  // 2^35 rows
    if (c->pages > 0 && (c->codes == nullptr || c->scales == nullptr || c->exponents == nullptr || !aligned16(c->codes) ||
                         !aligned16(c->scales) || !aligned16(c->exponents)))
        return DDGEMM_ERR_INVALID_ARG;
    int shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    v = CacheView{c->format, cache_width(c->head_dim), (int)c->head_dim, (int)c->heads, c->pages, (int)c->page_size, shift,
                  c->codes, c->scales, c->exponents};
    return DDGEMM_OK;
}

ddgemm_status check_batch(const ddgemm_batch* b, BatchView& v) {
    if (b == nullptr || b->tokens < 0 || b->batch < 0 || b->table_pages < 0) return DDGEMM_ERR_INVALID_ARG;
    if (b->tokens > DDGEMM_MAX_TOKENS || b->batch > DDGEMM_MAX_TOKENS || b->table_pages > DDGEMM_MAX_TOKENS)
        return DDGEMM_ERR_UNSUPPORTED;
    if (b->batch > 0 && b->tokens > 0) {
        if (b->starts == nullptr || b->lengths == nullptr || (b->page_table == nullptr && b->table_pages > 0)) return DDGEMM_ERR_INVALID_ARG;
        if (((uintptr_t)b->starts | (uintptr_t)b->lengths | (uintptr_t)b->page_table) % 4 != 0) return DDGEMM_ERR_INVALID_ARG;
        if (b->batch > 1 && b->table_stride < b->table_pages) return DDGEMM_ERR_INVALID_ARG;
    }
    v = BatchView{b->tokens, (int)b->batch, b->starts, b->lengths, b->page_table, (int)b->table_pages, b->table_stride};
    return DDGEMM_OK;
}

bool overlaps_cache(const CacheView& c, const void* p, int64_t bytes) {
    const int64_t rows = c.pages * 2 * c.heads * c.page_size;
    return overlap(c.codes, rows * (c.width / 2), p, bytes) || overlap(c.scales, rows * (c.width / mx4_block(c.fmt)), p, bytes) ||
           overlap(c.exponents, rows, p, bytes);
}
bool overlaps_batch(const BatchView& b, const void* p, int64_t bytes) {
    return overlap(b.starts, (b.batch + 1LL) * 4, p, bytes) || overlap(b.lengths, b.batch * 4LL, p, bytes) ||
           overlap(b.table, b.batch > 0 ? ((b.batch - 1) * b.ld_table + b.table_pages) * 4 : 0, p, bytes);
}
// Nothing of the cache or of the batch is written through another argument.
bool batch_in_cache(const CacheView& c, const BatchView& b) {
    return overlaps_cache(c, b.starts, (b.batch + 1LL) * 4) || overlaps_cache(c, b.lengths, b.batch * 4LL) ||
           overlaps_cache(c, b.table, b.batch > 0 ? ((b.batch - 1) * b.ld_table + b.table_pages) * 4 : 0);
}

// The factor of a rotation as a float and what it leaves.
void two_floats(double x, float& hi, float& lo) {
    hi = (float)x;
    lo = std::isfinite(hi) ? (float)(x - (double)hi) : 0.0f;
}

ddgemm_status check_rotary(const ddgemm_rotary* r, int64_t dim) {
    if (r == nullptr || r->pairs < 0 || (r->interleaved != 0 && r->interleaved != 1)) return DDGEMM_ERR_INVALID_ARG;
    if (r->pairs > dim / 2) return DDGEMM_ERR_INVALID_ARG;
    if (r->pairs > 0 && (r->turns == nullptr || (uintptr_t)r->turns % 8 != 0)) return DDGEMM_ERR_INVALID_ARG;
    return DDGEMM_OK;
}

// Rows (query tokens times heads of a group) of a sequence on average up to which the
// kernel for few queries runs: it reads the cache once for each 8 of them, the other
// once for 256.  Width 128, us, this kernel and the other: 32 sequences of 2048 to 4096
// tokens with 8 heads, 32 rows 119 and 153, 48 rows 168 and 157, 64 rows 218 and 156;
// one of 65536, 48 rows 105 and 118, 64 rows 132 and 116; one of 4096, 64 rows 24 and 23.
constexpr int64_t kColumnsMost = 48;
// The host knows the sum of the sequences' rows alone.  Where their average is more, or
// the tokens beyond one for each slot of the batch are more than 512 rows, both kernels run,
// each on its sequences.  127 single tokens and 128 of one further sequence, 4000 in the
// cache, 8 heads: 208 us, 299 by the kernel for few alone; 1024 of that sequence: 320 us,
// 706 by the other alone.  What it costs where no sequence has many: 32 of 5 tokens each
// 194 us, 172 by the kernel for few alone.  Slots without tokens hide a part from this rule:
// 255 tokens behind 4000, in 256 slots, are the kernel for few's, 353 us (112 in a slot of
// their own).  To run both wherever all tokens could be of one sequence takes 138 us there,
// but costs batches of single tokens more: 65 of 4000 105 us for 83, 1024 of 100 137 for 112.
constexpr int64_t kSurplus = 512;

ddgemm_status attend_tiles_call(AttendArgs& a, int type, cudaStream_t st) {
    a.splits = attend_tile_parts(a);
    if (a.above > 0) {  // every token has room in it, those of other sequences too: 256 MB at most
        const int64_t row = a.c.width * 4 + (int64_t)sizeof(float4), most = (256LL << 20) / (row * a.b.tokens * a.heads);
        a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(a.splits, most));
    }
    Workspace ws(st);
    const int64_t rows = a.splits > 1 ? a.splits * a.b.tokens * a.heads : 0;
    const int64_t parts = ws.reserve(rows * (int64_t)sizeof(float4)), sums = ws.reserve(rows * a.c.width * 4);
    if (!ws.allocate()) return DDGEMM_ERR_ALLOC;
    if (rows > 0) a.part = ws.at<float4>(parts), a.sums = ws.at<float>(sums);
    return status_of(launch_attend_tile(a, type, st));
}

ddgemm_status attend_columns_call(AttendArgs& a, int type, cudaStream_t st) {
    plan_attend_columns(a, type);
    Workspace ws(st);
    const int64_t rows = a.together ? 0 : attend_columns_rows(a.splits);
    const int64_t parts = ws.reserve(rows * (int64_t)sizeof(float4)), sums = ws.reserve(rows * a.c.width * 4),
                  cuts = ws.reserve(rows > 0 ? a.splits * (int64_t)sizeof(CutItem) : 0);
    if (!ws.allocate()) return DDGEMM_ERR_ALLOC;
    if (rows > 0) a.part = ws.at<float4>(parts), a.sums = ws.at<float>(sums), a.cuts = ws.at<CutItem>(cuts);
    return status_of(launch_attend_columns(a, type, st));
}

}  // namespace

extern "C" {

ddgemm_status dd_rotary(int type, int64_t tokens, int64_t heads, int64_t dim, const void* x, int64_t x_token,
                        int64_t x_head, const void* positions, int wide, const ddgemm_rotary* rotary, int inverse,
                        void* y, int64_t y_token, int64_t y_head, void* stream) {
    if (!known_type(type) || tokens < 0 || heads < 0 || dim < 0 || (wide != 0 && wide != 1) || (inverse != 0 && inverse != 1))
        return DDGEMM_ERR_INVALID_ARG;
    if (tokens > DDGEMM_MAX_TOKENS || heads > DDGEMM_MAX_HEADS || dim > DDGEMM_MAX_ROTARY_DIM) return DDGEMM_ERR_UNSUPPORTED;
    const ddgemm_status s = check_rotary(rotary, dim);
    if (s != DDGEMM_OK) return s;
    const Heads in{x, tokens, heads, dim, x_token, x_head, type_bytes(type)}, out{y, tokens, heads, dim, y_token, y_head, type_bytes(type)};
    if (!in.sound() || !out.sound()) return DDGEMM_ERR_INVALID_ARG;
    if (tokens == 0 || heads == 0 || dim == 0) return DDGEMM_OK;
    const int64_t pos = wide ? 8 : 4;
    if (positions == nullptr || (uintptr_t)positions % pos != 0) return DDGEMM_ERR_INVALID_ARG;
    const bool in_place = x == y && (tokens <= 1 || x_token == y_token) && (heads <= 1 || x_head == y_head);
    if (!in_place && meet(in, out)) return DDGEMM_ERR_INVALID_ARG;
    if (overlap(positions, tokens * pos, y, out.bytes()) || overlap(rotary->turns, rotary->pairs * 8, y, out.bytes()))
        return DDGEMM_ERR_INVALID_ARG;
    Rotary r{type, tokens, (int)heads, (int)dim, x, x_token, x_head, y, y_token, y_head, positions, wide == 1, rotary->turns,
             (int)rotary->pairs, 0.0f, 0.0f, rotary->interleaved == 1, inverse == 1, 0};
    two_floats(rotary->scale, r.m, r.ml);
    return status_of(launch_rotary(r, static_cast<cudaStream_t>(stream)));
}

ddgemm_status dd_mx4_cache_layout(int format, int64_t head_dim, int64_t* width, int64_t* scale_bytes) {
    if (!known_format(format) || head_dim < 1) return DDGEMM_ERR_INVALID_ARG;
    if (head_dim > 256) return DDGEMM_ERR_UNSUPPORTED;
    const int w = cache_width(head_dim);
    if (width) *width = w;
    if (scale_bytes) *scale_bytes = w / mx4_block(format);
    return DDGEMM_OK;
}

ddgemm_status dd_mx4_cache_append(const ddgemm_mx4_cache* cache, const ddgemm_batch* batch, int type, const void* k,
                                  int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                                  const ddgemm_rotary* rotary, void* stream) {
    CacheAppend g{};
    if (!known_type(type)) return DDGEMM_ERR_INVALID_ARG;
    ddgemm_status s = check_cache(cache, g.cache);
    if (s == DDGEMM_OK) s = check_batch(batch, g.batch);
    if (s == DDGEMM_OK && rotary != nullptr) s = check_rotary(rotary, cache->head_dim);
    if (s != DDGEMM_OK) return s;
    const int64_t T = batch->tokens, H = cache->heads, D = cache->head_dim;
    const Heads hk{k, T, H, D, k_token, k_head, type_bytes(type)}, hv{v, T, H, D, v_token, v_head, type_bytes(type)};
    if (!hk.sound() || !hv.sound()) return DDGEMM_ERR_INVALID_ARG;
    if (T == 0 || batch->batch == 0) return DDGEMM_OK;
    if (overlaps_cache(g.cache, k, hk.bytes()) || overlaps_cache(g.cache, v, hv.bytes()) || batch_in_cache(g.cache, g.batch) ||
        (rotary != nullptr && overlaps_cache(g.cache, rotary->turns, rotary->pairs * 8)))
        return DDGEMM_ERR_INVALID_ARG;
    g.type = type;
    g.k = k, g.kt = k_token, g.kh = k_head;
    g.v = v, g.vt = v_token, g.vh = v_head;
    if (rotary != nullptr && rotary->pairs > 0) {
        g.turns = rotary->turns;
        g.half = (int)rotary->pairs;
        two_floats(rotary->scale, g.m, g.ml);
        g.interleaved = rotary->interleaved == 1;
    }
    return status_of(launch_cache_append(g, static_cast<cudaStream_t>(stream)));
}

ddgemm_status dd_mx4_cache_read(const ddgemm_mx4_cache* cache, const ddgemm_batch* batch, int type, void* k,
                                int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head, void* stream) {
    CacheRead g{};
    if (!known_type(type)) return DDGEMM_ERR_INVALID_ARG;
    ddgemm_status s = check_cache(cache, g.cache);
    if (s == DDGEMM_OK) s = check_batch(batch, g.batch);
    if (s != DDGEMM_OK) return s;
    const int64_t T = batch->tokens, H = cache->heads, D = cache->head_dim;
    const Heads hk{k, T, H, D, k_token, k_head, type_bytes(type)}, hv{v, T, H, D, v_token, v_head, type_bytes(type)};
    if (!hk.sound() || !hv.sound()) return DDGEMM_ERR_INVALID_ARG;
    if (T == 0 || batch->batch == 0) return DDGEMM_OK;
    if (meet(hk, hv)) return DDGEMM_ERR_INVALID_ARG;
    for (const Heads* h : {&hk, &hv})
        if (overlaps_cache(g.cache, h->p, h->bytes()) || overlaps_batch(g.batch, h->p, h->bytes())) return DDGEMM_ERR_INVALID_ARG;
    g.type = type;
    g.k = k, g.kt = k_token, g.kh = k_head;
    g.v = v, g.vt = v_token, g.vh = v_head;
    return status_of(launch_cache_read(g, static_cast<cudaStream_t>(stream)));
}

ddgemm_status dd_mx4_attention(const ddgemm_mx4_cache* cache, const ddgemm_batch* batch, int type, int64_t q_heads,
                               const void* q, int64_t q_token, int64_t q_head, int64_t window, int64_t sinks,
                               float scale, void* out, int64_t out_token, int64_t out_head, void* stream) {
    AttendArgs a{};
    if (!known_type16(type) || window < 0 || sinks < 0) return DDGEMM_ERR_INVALID_ARG;
    ddgemm_status s = check_cache(cache, a.c);
    if (s == DDGEMM_OK) s = check_batch(batch, a.b);
    if (s != DDGEMM_OK) return s;
    if (q_heads < 1 || q_heads % cache->heads != 0) return DDGEMM_ERR_INVALID_ARG;
    if (q_heads > DDGEMM_MAX_HEADS) return DDGEMM_ERR_UNSUPPORTED;
    const int64_t T = batch->tokens, D = cache->head_dim;
    const Heads hq{q, T, q_heads, D, q_token, q_head, 2}, ho{out, T, q_heads, D, out_token, out_head, 2};
    if (!hq.sound() || !ho.sound()) return DDGEMM_ERR_INVALID_ARG;
    if (T == 0 || batch->batch == 0) return DDGEMM_OK;
    if (meet(hq, ho) || overlaps_cache(a.c, out, ho.bytes()) || overlaps_batch(a.b, out, ho.bytes())) return DDGEMM_ERR_INVALID_ARG;
    a.q = q, a.qt = q_token, a.qh = q_head;
    a.out = out, a.ot = out_token, a.oh = out_head;
    a.heads = (int)q_heads;
    a.group = (int)(q_heads / cache->heads);
    const int64_t far = (1LL << 31) - 65536;  // a window or sinks of so many leave nothing out
    a.window = window < far && sinks < far ? (int)window : 0;
    a.sinks = a.window > 0 ? (int)sinks : 0;
    a.scale = scale * 1.4426950408889634f;
    if (!std::isfinite(a.scale)) return DDGEMM_ERR_INVALID_ARG;
    const auto whole = [&](const void* p, int64_t t, int64_t h) { return aligned16(p) && (T <= 1 || t % 8 == 0) && (q_heads <= 1 || h % 8 == 0); };
    a.vec_q = whole(q, q_token, q_head);
    a.vec_out = whole(out, out_token, out_head);
    if (a.tiles(8) * cache->heads >= (1LL << 31) || T * a.group >= (1LL << 31)) return DDGEMM_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t rows = T * a.group, surplus = (T - batch->batch) * a.group;
    const bool tiles = cache->pages > 0 && (rows > kColumnsMost * batch->batch || surplus > kSurplus);
    const bool columns = !tiles || (batch->batch > 1 && a.group <= kColumnsMost);
    a.above = 0, a.upto = INT64_MAX;
    for (const bool tile : {false, true}) {
        if (!(tile ? tiles : columns)) continue;
        AttendArgs c = a;
        if (tile && columns) {
            c.above = kColumnsMost;
            const int64_t step = kColumnsMost / a.group + 1;
            if (T / step < batch->batch) c.step = (int)step;
        }
        if (!tile && tiles) c.upto = kColumnsMost;
        s = tile ? attend_tiles_call(c, type, st) : attend_columns_call(c, type, st);
        if (s != DDGEMM_OK) return s;
    }
    return DDGEMM_OK;
}

}  // extern "C"
