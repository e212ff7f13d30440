// Host side of lso_orthogonalize and lso_muon_step: checks, the workspace
// plan and the table of a call.
#include <algorithm>
#include <cmath>
#include <new>
#include <utility>
#include <vector>

#include "lso_ns.h"
#include "lso_ops.h"
#include "lso_runtime.h"

namespace lso {
namespace {

constexpr uint64_t kMaxSide = (1ull << 31) - 1;
constexpr uint64_t kMaxIndex = (1ull << 23) - 8;   // workgroups of a launch: up to 512 lanes each, under 2^32 in all
constexpr double kDefaultCoef[3] = {3.4445, -4.7750, 2.0315};

// A matrix of either call, before its place in the plan.
struct Item {
    NsMat mat;
    uint64_t rows, cols;
};

uint64_t padded(uint64_t n, uint64_t tile) { return (n + tile - 1) / tile * tile; }

// The largest smaller side that takes the small path: 64, but 32 where the
// launches of the general path are made anyway, for larger matrices, and
// those of 33 to 64 have less than kApart elements along their long sides.
// Measured (us, with the general path for those / apart from it): 6 of
// 1024 x 1024 with 4, 16, 32 and 64 of 64 x 2048 672 / 746, 719 / 748, 784 / 756, 918 / 791;
// one of 100 x 100 with 16, 32 and 64 of them 138 / 161, 162 / 168, 240 / 200.
constexpr uint64_t kApart = 65536;

uint64_t small_side(const std::vector<Item>& items)
{
    bool larger = false;
    uint64_t length = 0;
    for (const Item& it : items) {
        const uint64_t k = std::min(it.rows, it.cols);
        if (k > LSO_NS_SMALL_SIDE) larger = true;
        else if (k > 32) length += std::max(it.rows, it.cols);
    }
    return larger && length < kApart ? 32 : LSO_NS_SMALL_SIDE;
}

// Which of the small path's kernels, -1 for none.
int small_class(uint64_t k, uint64_t side) { return k > side ? -1 : k <= 8 ? 0 : k <= 16 ? 1 : k <= 32 ? 2 : 3; }

// The largest values that a run from s <= 1 can meet: of the iterates'
// singular values s, of s^2 and of the polynomial a + b s^2 + c s^4; and for
// each step the power of two that the polynomial stays under, and whether it
// and the next step's may be multiplied with each other (and with S).
double most_value(const double* coef, uint32_t steps, int16_t* shift, bool* pair)
{
    double s = 1.0, most = 1.0, poly_before = 0.0;
    bool alone = false;
    for (uint32_t k = 0; k < steps; ++k) {
        const double a = coef[3 * k], b = coef[3 * k + 1], c = coef[3 * k + 2], z = s * s;
        double poly = std::max(std::fabs(a), std::fabs(a + b * z + c * z * z));
        if (c != 0.0 && -b / (2 * c) > 0.0 && -b / (2 * c) < z) poly = std::max(poly, std::fabs(a - b * b / (4 * c)));
        most = std::max({most, z, poly});
        if (k > 0) pair[k - 1] = !alone && poly_before * poly <= kNsMostValue;
        alone = !(poly * z <= kNsMostValue);
        poly_before = poly;
        pair[k] = false;
        int above = 0;
        if (poly > 0.0 && poly <= kNsMostValue) (void)std::frexp(poly, &above);
        shift[k] = static_cast<int16_t>(std::max(above, -255));
        // s p(s^2) on [0, s]: at the end, and where 5 c t^2 + 3 b t + a = 0, t = s^2
        auto value = [&](double t) { return std::sqrt(t) * std::fabs(a + t * (b + t * c)); };
        double next = value(z);
        const double disc = 9 * b * b - 20 * a * c;
        if (c != 0.0 && disc >= 0.0) {
            for (const double t : {(-3 * b + std::sqrt(disc)) / (10 * c), (-3 * b - std::sqrt(disc)) / (10 * c)})
                if (t > 0.0 && t < z) next = std::max(next, value(t));
        } else if (c == 0.0 && b != 0.0) {
            const double t = -a / (3 * b);
            if (t > 0.0 && t < z) next = std::max(next, value(t));
        }
        s = next;
        most = std::max(most, s);
    }
    return most;
}

lso_status check_params(const lso_ns_params* p, NsCall& c)
{
    c.steps = p ? p->steps : 5;
    c.eps = p ? p->eps : 1e-7;
    if (p && p->precision > LSO_NS_HALF) return fail(LSO_E_INVALID, "unknown precision %u", p->precision);
    if (c.steps < 1 || c.steps > LSO_NS_MAX_STEPS)
        return fail(LSO_E_INVALID, "steps must be 1 to %u (got %u)", LSO_NS_MAX_STEPS, c.steps);
    if (!(std::isfinite(c.eps) && c.eps >= 0.0)) return fail(LSO_E_INVALID, "eps must be finite and >= 0");
    for (uint32_t k = 0; k < 3 * c.steps; ++k) {
        c.coef[k] = p && p->coef ? p->coef[k] : kDefaultCoef[k % 3];
        if (!std::isfinite(c.coef[k])) return fail(LSO_E_INVALID, "coefficient %u is not finite", k);
    }
    const double most = most_value(c.coef, c.steps, c.shift, c.pair);
    if (!(most <= kNsMostValue))
        return fail(LSO_E_INVALID, "the coefficients let a value reach %.3g, more than %.3g", most, kNsMostValue);
    return LSO_OK;
}

// Bytes from the first to the last element of rows x cols at stride ld.
uint64_t span(uint64_t rows, uint64_t cols, uint64_t ld, uint64_t elem) { return ((rows - 1) * ld + cols) * elem; }

// kNsQuads if the matrix may be read and written four columns at a time.
uint32_t quads(const NsMat& m, uint64_t cols)
{
    auto fits = [](const void* p, uint64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    const bool ok = cols % 4 == 0 && m.ld_src % 4 == 0 && m.ld_dst % 4 == 0 && fits(m.src, (m.flags & kNsSrcF32) ? 16 : 8) &&
                    fits(m.dst, (m.flags & kNsDstF32) ? 16 : 8) && fits(m.m, 16) && fits(m.master, 16);
    return ok ? kNsQuads : 0;
}

lso_status check_sides(uint64_t rows, uint64_t cols, size_t i)
{
    if (rows > kMaxSide || cols > kMaxSide) return fail(LSO_E_INVALID, "matrix %zu: a side is too large", i);
    if (rows != 0 && cols > (1ull << 56) / rows) return fail(LSO_E_INVALID, "matrix %zu: too many elements", i);
    return LSO_OK;
}

lso_status take_array(std::vector<Interval>& iv, uintptr_t addr, uint64_t bytes, uint64_t elem, bool written, size_t i,
                      const char* name)
{
    if (addr == 0) return fail(LSO_E_INVALID, "matrix %zu: %s address is NULL", i, name);
    if (addr % elem != 0) return fail(LSO_E_ALIGN, "matrix %zu: %s is not aligned to its elements", i, name);
    if (!add_array(iv, addr, bytes, written, i))
        return fail(LSO_E_INVALID, "matrix %zu: %s range wraps the address space", i, name);
    return LSO_OK;
}

// The arrays of a call by kind: those of a kind mostly lie in order, so their
// check sorts little.
struct Arrays {
    std::vector<Interval> kind[4];

    std::vector<Interval> all()
    {
        std::vector<Interval> iv;
        iv.reserve(kind[0].size() + kind[1].size() + kind[2].size() + kind[3].size() + 1);
        for (const auto& k : kind) {
            const size_t at = iv.size();
            iv.insert(iv.end(), k.begin(), k.end());
            const auto below = [](const Interval& a, const Interval& b) { return a.lo < b.lo; };
            if (!std::is_sorted(iv.begin() + at, iv.end(), below)) std::sort(iv.begin() + at, iv.end(), below);
            std::inplace_merge(iv.begin(), iv.begin() + at, iv.end(), below);
        }
        return iv;
    }
};

// The checks of lso_orthogonalize; with arrays, of its addresses too.
lso_status collect(const lso_matrix* mats, size_t n, std::vector<Item>& items, Arrays* arrays)
{
    if (n > 0 && !mats) return fail(LSO_E_INVALID, "mats is NULL");
    for (size_t i = 0; i < n; ++i) {
        const lso_matrix& a = mats[i];
        for (const uint32_t d : {a.x_dtype, a.y_dtype})
            if (d != LSO_DT_F32 && d != LSO_DT_BF16)
                return fail(LSO_E_DTYPE, "matrix %zu: x and y must be F32 or BF16", i);
        lso_status s = check_sides(a.rows, a.cols, i);
        if (s != LSO_OK) return s;
        if (a.rows == 0 || a.cols == 0) continue;
        if (a.ld_x < a.cols || a.ld_y < a.cols || a.ld_x > kMaxSide || a.ld_y > kMaxSide)
            return fail(LSO_E_INVALID, "matrix %zu: a row stride is smaller than cols, or too large", i);
        const uint64_t ex = a.x_dtype == LSO_DT_F32 ? 4 : 2, ey = a.y_dtype == LSO_DT_F32 ? 4 : 2;
        if (arrays) {
            const bool same = a.x == a.y && a.x_dtype == a.y_dtype && a.ld_x == a.ld_y;
            if (!same) {
                s = take_array(arrays->kind[0], reinterpret_cast<uintptr_t>(a.x), span(a.rows, a.cols, a.ld_x, ex), ex, false, i, "x");
                if (s != LSO_OK) return s;
            }
            s = take_array(arrays->kind[1], reinterpret_cast<uintptr_t>(a.y), span(a.rows, a.cols, a.ld_y, ey), ey, true, i, "y");
            if (s != LSO_OK) return s;
        }
        Item it{};
        it.rows = a.rows;
        it.cols = a.cols;
        it.mat.src = a.x;
        it.mat.dst = a.y;
        it.mat.ld_src = static_cast<uint32_t>(a.ld_x);
        it.mat.ld_dst = static_cast<uint32_t>(a.ld_y);
        it.mat.flags = (a.x_dtype == LSO_DT_F32 ? kNsSrcF32 : 0) | (a.y_dtype == LSO_DT_F32 ? kNsDstF32 : 0);
        it.mat.flags |= quads(it.mat, it.cols);
        items.push_back(it);
    }
    return LSO_OK;
}

lso_status collect(const lso_muon_block* blocks, size_t n, std::vector<Item>& items, Arrays* arrays)
{
    if (n > 0 && !blocks) return fail(LSO_E_INVALID, "blocks is NULL");
    for (size_t i = 0; i < n; ++i) {
        const lso_muon_block& b = blocks[i];
        if (b.grad_dtype != LSO_DT_BF16 && b.grad_dtype != LSO_DT_F32)
            return fail(LSO_E_DTYPE, "matrix %zu: gradient dtype must be BF16 or F32", i);
        if (b.weight_dtype != LSO_DT_BF16 && b.weight_dtype != LSO_DT_NONE)
            return fail(LSO_E_DTYPE, "matrix %zu: weight dtype must be BF16 or NONE", i);
        if ((b.flags & ~LSO_MUON_NESTEROV) != 0 || b.reserved != 0)
            return fail(LSO_E_INVALID, "matrix %zu: unknown flags or reserved field", i);
        if (!std::isfinite(b.lr) || !std::isfinite(b.weight_decay) || !std::isfinite(b.scale))
            return fail(LSO_E_INVALID, "matrix %zu: lr, weight_decay and scale must be finite", i);
        if (!(b.beta >= 0.0 && b.beta < 1.0)) return fail(LSO_E_INVALID, "matrix %zu: beta must be in [0, 1)", i);
        lso_status s = check_sides(b.rows, b.cols, i);
        if (s != LSO_OK) return s;
        if (b.rows == 0 || b.cols == 0) continue;
        const uintptr_t base = reinterpret_cast<uintptr_t>(b.base);
        const uint64_t count = b.rows * b.cols, eg = b.grad_dtype == LSO_DT_F32 ? 4 : 2;
        const bool weight = b.weight_dtype == LSO_DT_BF16;
        if (arrays) {
            const struct { uint64_t off, elem; bool used, written; const char* name; } arr[4] = {
                {b.off_master, 4, true, true, "master"},
                {b.off_m, 4, true, true, "m"},
                {b.off_grad, eg, true, false, "grad"},
                {b.off_weight, 2, weight, true, "weight"},
            };
            for (size_t k = 0; k < 4; ++k) {
                const auto& a = arr[k];
                if (!a.used) continue;
                s = take_array(arrays->kind[k], base + a.off, count * a.elem, a.elem, a.written, i, a.name);
                if (s != LSO_OK) return s;
            }
        }
        Item it{};
        it.rows = b.rows;
        it.cols = b.cols;
        it.mat.src = reinterpret_cast<const void*>(base + b.off_grad);
        it.mat.dst = weight ? reinterpret_cast<void*>(base + b.off_weight) : nullptr;
        it.mat.m = reinterpret_cast<float*>(base + b.off_m);
        it.mat.master = reinterpret_cast<float*>(base + b.off_master);
        it.mat.ld_src = it.mat.ld_dst = static_cast<uint32_t>(b.cols);
        it.mat.flags = kNsMuon | (eg == 4 ? kNsSrcF32 : 0) | ((b.flags & LSO_MUON_NESTEROV) ? kNsNesterov : 0);
        it.mat.beta = static_cast<float>(b.beta);
        it.mat.c1 = static_cast<float>(1.0 - b.beta);
        it.mat.keep = static_cast<float>(1.0 - b.lr * b.weight_decay);
        it.mat.step = static_cast<float>(-b.lr * b.scale);
        if (!std::isfinite(it.mat.keep) || !std::isfinite(it.mat.step))
            return fail(LSO_E_INVALID, "matrix %zu: lr * weight_decay or lr * scale is not an FP32 number", i);
        it.mat.flags |= quads(it.mat, it.cols);
        items.push_back(it);
    }
    return LSO_OK;
}

// How the products of the general path are cut up.  A launch should give
// each of the GPU's 256 CUs the same work: `slots` workgroups run at a time,
// so the tiles' summed index is cut into parts of `depth` stages such that
// the parts fill a whole number of rounds of slots; the cost of a round is its
// depth plus kPartCost stages (filling the pipeline, storing and adding up
// the sums).
struct Tiles {
    uint64_t count, stages;   // of one matrix in one launch
    uint64_t matrices;        // so many with the same numbers
};
// kPartCost: measured over calls of one to four matrices of 64 x 2048 to 4096 x 4096:
// 8 and 16 cut too finely (1024 x 1024 half precision 243 against 178 us with
// 64), 32 and 128 are within 3% of 64.
constexpr uint64_t kPartCost = 64;

uint64_t units_of(const std::vector<Tiles>& list, uint64_t depth)
{
    uint64_t units = 0;
    for (const Tiles& t : list) units += t.matrices * ((t.count * ((t.stages + depth - 1) / depth) + 7) / 8 * 8);
    return units;
}

uint32_t part_depth(const std::vector<Tiles>& matrices, uint64_t slots)
{
    std::vector<Tiles> list;   // equal ones, which mostly lie in a row, together
    uint64_t most = 1;
    for (const Tiles& t : matrices) {
        most = std::max(most, t.stages);
        if (!list.empty() && list.back().count == t.count && list.back().stages == t.stages) ++list.back().matrices;
        else list.push_back(t);
    }
    const uint64_t whole_units = units_of(list, most);
    if (whole_units > 8 * slots) return static_cast<uint32_t>(most);   // many rounds: nothing to gain
    uint64_t best = most, best_cost = (whole_units + slots - 1) / slots * (most + kPartCost / 2);
    for (uint64_t depth = most - 1; depth >= 8; --depth) {
        const uint64_t units = units_of(list, depth);
        if (units > 8 * slots) break;
        // the smallest depth with as many parts of each matrix: as many units,
        // and the cheapest (trying each depth took 11 ms for 40 x 2^26)
        uint64_t same = 8;
        for (const Tiles& t : list) {
            const uint64_t parts = (t.stages + depth - 1) / depth;
            same = std::max(same, (t.stages + parts - 1) / parts);
        }
        depth = std::min(depth, same);
        const uint64_t cost = (units + slots - 1) / slots * (depth + kPartCost);
        if (cost < best_cost) {
            best = depth;
            best_cost = cost;
        }
    }
    return static_cast<uint32_t>(best);
}

// The index of `count` matrices in a launch of `total` workgroups, by the first
// one that each has.
NsIndex index_of(const NsMat* mats, uint32_t count, uint32_t NsMat::*first, uint32_t total)
{
    NsIndex x{};
    for (uint32_t i = 0; i < count; ++i) {
        const uint32_t each = (i + 1 < count ? mats[i + 1].*first : total) - mats[i].*first;
        if (x.runs > 0 && x.each[x.runs - 1] == each) continue;
        if (x.runs == kNsRuns) {
            x.runs = 0;
            return x;
        }
        x.first[x.runs] = mats[i].*first;
        x.first_mat[x.runs] = i;
        x.each[x.runs] = each;
        ++x.runs;
    }
    return x;
}

// Whether to take steps in pairs, by the matrix-core products of two steps: a
// pair has seven launches instead of six, so small calls need a larger saving.
bool pairs_pay(uint32_t edge, double single, double pair) { return pair * (edge == 64 ? 1.4 : 1.1) < single; }

// The edge of the products' tiles.  Large tiles load less per operation; small
// ones fill the 256 CUs with less work, waste less on padding and on the upper
// half of diagonal tiles, and fill and drain their pipeline sooner.  The edge
// is the one whose launches of five steps cost least: a tile costs its stages
// and `tile` more, a launch `launch` stages of latency, and `slots` workgroups
// take `us` for a stage.  The numbers are fitted to 100 measured calls, one
// to 200 matrices of 100 x 2000 to 8192 x 8192 in both precisions, whose time is
// 1.2% over the best edge's in the mean and 11% at most (a rule by the operations
// of a step alone: 2.3% and 29%).  Measured (us, edges 64 / 128 / 256): 22 of
// 256 x 2048 in half precision 301 / 383 / 600; in full precision 200 of 300 x 900 2264 /
// 2910 / 6726, 2048 x 2048 850 / 777 / 1349, the seven of a TinyLlama layer 5977 / 4003 /
// 4220, three of 4096 x 4096 15106 / 11164 / 10441.
uint32_t tile_edge(const std::vector<Item>& items, uint64_t side, double single, double pair)
{
    constexpr struct { uint32_t edge; double slots, tile, launch, us; } edges[3] = {
        {64, 1024, 32, 24, 0.29}, {128, 512, 80, 80, 0.286}, {256, 256, 128, 160, 0.4}};
    uint32_t best = 64;
    double best_cost = INFINITY;
    for (const auto& x : edges) {
        // launches with S, with the other squares and with X
        const bool pairs = pairs_pay(x.edge, single, pair);
        const double grams = pairs ? 3 : 5, squares = pairs ? 11 : 5, applies = pairs ? 3 : 5;
        double stages = 0.0;
        for (const Item& it : items) {
            const uint64_t k = std::min(it.rows, it.cols), l = std::max(it.rows, it.cols);
            if (k <= side) continue;
            const double tm = static_cast<double>((k + x.edge - 1) / x.edge), tn = static_cast<double>((l + x.edge - 1) / x.edge);
            const double half = tm * (tm + 1) / 2, m = tm * x.edge / 16 + x.tile, n = tn * x.edge / 16 + x.tile;
            stages += grams * half * n + squares * half * m + applies * tm * tn * m;
        }
        const double cost = x.us * (stages / x.slots + (grams + squares + applies) * x.launch);
        if (cost < best_cost) {
            best = x.edge;
            best_cost = cost;
        }
    }
    return best;
}

// How the call's numbers are held, its tiles' edge, and whether steps are taken in pairs:
// X_{k+2} = Q X_k with Q = P' P, P' the polynomial in S' = P S P.  A step by
// itself makes S = X X^T (half of it, m^2 n operations), S^2 (m^3) and P X (2 m^2 n); a
// pair makes S, Q X and five products of m x m, so it saves 3 m^2 n - 3 m^3
// of 6 m^2 n + 2 m^3.  It loses no accuracy: S' is as far from the product of
// the next X with itself as rounding makes that one.  In half precision the
// squares keep two terms then (with one the error grows, with two it falls
// below that of single steps), which costs three products for each one.
// The plan depends on sizes and precision alone, not on the steps: so does the
// workspace.  Measured: 8192 x 28672 58.0 against 77.3 ms, the seven
// matrices of a TinyLlama layer 4.30 against 5.00 ms (both with tiles of 256).
NsLayout layout_of(const lso_ns_params* p, const std::vector<Item>& items, NsCall& c)
{
    const uint32_t terms = p && p->precision == LSO_NS_HALF ? 1 : 2;
    const uint64_t side = small_side(items);
    double single = 0.0, pair = 0.0;   // matrix-core products of two steps
    for (const Item& it : items) {
        const double m = static_cast<double>(std::min(it.rows, it.cols)), n = static_cast<double>(std::max(it.rows, it.cols));
        if (std::min(it.rows, it.cols) <= side) continue;
        single += terms == 2 ? 3 * (6 * m * m * n + 2 * m * m * m) : 10 * m * m * n + 2 * m * m * m;
        pair += terms == 2 ? 3 * (3 * m * m * n + 5 * m * m * m) : 5 * m * m * n + 15 * m * m * m;
    }
    c.tile = tile_edge(items, side, single, pair);
    c.pairs = pairs_pay(c.tile, single, pair);
    return c.pairs ? NsLayout{terms, 2, 4} : NsLayout{terms, terms, 2};
}

// Order the items (small path by class, then the general path, deep matrices
// first), give each its part of the workspace and its first index in every
// launch.  work is the workspace's address (0 to plan only); returns the
// bytes needed, the table's first, or 0 with an error set.
uint64_t plan(std::vector<Item>& items, NsCall& c, uintptr_t work, std::vector<NsMat>& table)
{
    uint64_t at = (items.size() * sizeof(NsMat) + 255) / 256 * 256;
    table.clear();
    table.reserve(items.size());
    // a launch ends sooner if the longest units start first
    const auto longer = [](const Item& a, const Item& b) { return std::max(a.rows, a.cols) > std::max(b.rows, b.cols); };
    if (!std::is_sorted(items.begin(), items.end(), longer)) {
        std::vector<std::pair<uint64_t, uint32_t>> order;   // longest first, then as given
        order.reserve(items.size());
        for (uint32_t i = 0; i < items.size(); ++i) order.push_back({UINT64_MAX - std::max(items[i].rows, items[i].cols), i});
        std::sort(order.begin(), order.end());
        std::vector<Item> sorted;
        sorted.reserve(items.size());
        for (const auto& o : order) sorted.push_back(items[o.second]);
        items.swap(sorted);
    }
    const uint64_t edge = c.tile, side = small_side(items);
    std::vector<Tiles> lists[4];
    uint64_t most_index = 0;
    for (int cls = 0; cls <= kNsClasses; ++cls) {
        uint64_t chunks = 0, prep = 0;
        uint32_t count = 0;
        for (const Item& it : items) {
            const uint64_t k = std::min(it.rows, it.cols), l = std::max(it.rows, it.cols);
            const int own = small_class(k, side);
            if ((own < 0 ? kNsClasses : own) != cls) continue;
            NsMat m = it.mat;
            m.rows = static_cast<uint32_t>(it.rows);
            m.cols = static_cast<uint32_t>(it.cols);
            if (it.rows > it.cols) m.flags |= kNsTall;
            m.work = reinterpret_cast<char*>(work + at);
            if (own >= 0) {
                m.prep0 = static_cast<uint32_t>(chunks);
                chunks += (l + kNsSmallChunk - 1) / kNsSmallChunk;
                at += ns_small_bytes(k, l);
            } else {
                const uint64_t mp = padded(k, edge), np = padded(l, edge), tm = mp / edge, tn = np / edge;
                if (mp > (1u << 20) || np > kMaxSide / 4) {
                    fail(LSO_E_INVALID, "a matrix of %llu x %llu is too large", static_cast<unsigned long long>(it.rows),
                         static_cast<unsigned long long>(it.cols));
                    return 0;
                }
                m.mp = static_cast<uint32_t>(mp);
                m.np = static_cast<uint32_t>(np);
                m.prep0 = static_cast<uint32_t>(prep);
                prep += mp / kNsPrep * (np / kNsPrep);
                at += ns_work(mp, np, c.layout).bytes;
                // a stage is so many blocks of 16 values of the summed index, of
                // 32 where both operands have one term
                const uint64_t gram = 16 * (3 - c.layout.x_terms) * ns_blocks(c.tile, true, c.layout.x_terms);
                const uint64_t square = 16 * (3 - c.layout.square_terms) * ns_blocks(c.tile, true, c.layout.square_terms);
                lists[0].push_back({tm * (tm + 1) / 2, np / gram, 1});
                lists[1].push_back({tm * (tm + 1) / 2, mp / square, 1});
                lists[2].push_back({tm * tn, mp / 16, 1});
                lists[3].push_back({tm * tn, mp / 32, 1});
            }
            ++count;
            most_index = std::max({most_index, chunks, prep, uint64_t{count} * 2});
            table.push_back(m);
        }
        if (cls < kNsClasses) {
            c.nsmall[cls] = count;
            c.small_chunks[cls] = static_cast<uint32_t>(chunks);
            c.small_index[cls] = index_of(table.data() + (table.size() - count), count, &NsMat::prep0, c.small_chunks[cls]);
        } else {
            c.nbig = count;
            c.prep_tiles = static_cast<uint32_t>(prep);
            c.prep_index = index_of(table.data() + (table.size() - count), count, &NsMat::prep0, c.prep_tiles);
        }
    }
    if (c.nbig > 0) {
        NsProduct* products[4] = {&c.gram, &c.square, &c.apply, &c.apply_one};
        uint32_t NsMat::*firsts[4] = {&NsMat::gram0, &NsMat::square0, &NsMat::apply0, &NsMat::apply_one0};
        uint64_t most_units = 0, part_units = 0;
        for (int p = 0; p < 4; ++p) {
            const uint64_t units_before = units_of(lists[p], UINT32_MAX);
            if (units_before > kMaxIndex) {
                most_index = units_before;
                break;
            }
            // as many workgroups as fit the LDS of the 256 CUs
            const bool two = ns_blocks(c.tile, p < 2, p == 0 ? c.layout.x_terms : c.layout.square_terms) == 2;
            products[p]->depth = part_depth(lists[p], edge == 256 ? 256 : edge == 128 || two ? 512 : 1024);
            uint64_t units = 0;
            bool cut = false;
            NsMat* m = table.data() + (table.size() - c.nbig);
            for (const Tiles& t : lists[p]) {
                const uint64_t parts = (t.stages + products[p]->depth - 1) / products[p]->depth;
                (m++)->*firsts[p] = static_cast<uint32_t>(units);
                units += (t.count * parts + 7) / 8 * 8;
                cut = cut || parts > 1;
            }
            products[p]->units = static_cast<uint32_t>(units);
            products[p]->index = index_of(table.data() + (table.size() - c.nbig), c.nbig, firsts[p], products[p]->units);
            most_units = std::max(most_units, units);
            if (cut) part_units = std::max(part_units, units);
        }
        most_index = std::max(most_index, most_units);
        c.counters = reinterpret_cast<uint32_t*>(work + at);
        c.ncounters = static_cast<uint32_t>(part_units);
        at += (part_units * 4 + 255) / 256 * 256;
        c.parts = reinterpret_cast<float*>(work + at);
        at += part_units * edge * edge * 4;
    }
    if (most_index > kMaxIndex) {
        fail(LSO_E_INVALID, "the call is too large: split it");
        return 0;
    }
    return at;
}


template <typename T>
uint64_t workspace_bytes(const T* list, size_t n, const lso_ns_params* params)
{
    clear_error();
    NsCall c{};
    std::vector<Item> items;
    std::vector<NsMat> table;
    if (check_params(params, c) != LSO_OK || collect(list, n, items, nullptr) != LSO_OK) return 0;
    c.layout = layout_of(params, items, c);
    return plan(items, c, 0, table);
}

template <typename T>
lso_status run(const T* list, size_t n, const lso_ns_params* params, void* workspace, uint64_t bytes, void* stream)
{
    clear_error();
    NsCall c{};
    std::vector<Item> items;
    std::vector<NsMat> table;
    Arrays arrays;
    items.reserve(n < 65536 ? n : 65536);
    lso_status s = check_params(params, c);
    if (s == LSO_OK) s = collect(list, n, items, &arrays);
    if (s != LSO_OK) return s;
    if (items.empty()) return LSO_OK;
    c.layout = layout_of(params, items, c);
    if (!workspace) return fail(LSO_E_INVALID, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return fail(LSO_E_ALIGN, "workspace must be 16-byte aligned");
    const uint64_t need = plan(items, c, reinterpret_cast<uintptr_t>(workspace), table);
    if (need == 0) return LSO_E_INVALID;
    if (bytes < need)
        return fail(LSO_E_INVALID, "workspace of %llu bytes is smaller than the %llu this call needs",
                    static_cast<unsigned long long>(bytes), static_cast<unsigned long long>(need));
    std::vector<Interval> iv = arrays.all();
    if (!add_array(iv, reinterpret_cast<uintptr_t>(workspace), need, true, n))
        return fail(LSO_E_INVALID, "workspace range wraps the address space");
    s = check_overlap(iv);
    if (s != LSO_OK) return s;
    c.table = table.data();
    const int err = ns_launch(c, static_cast<NsMat*>(workspace), stream);
    return err == 0 ? LSO_OK : hip_fail(err, "Newton-Schulz launch");
}

// std::bad_alloc does not cross the ABI.
template <typename F, typename R>
R guarded(F f, R none)
{
    try {
        return f();
    } catch (const std::exception& e) {
        fail(LSO_E_NOMEM, "host memory: %s", e.what());
        return none;
    }
}

}  // namespace
}  // namespace lso

extern "C" {

uint64_t lso_orthogonalize_workspace_bytes(const lso_matrix* mats, size_t n, const lso_ns_params* params)
{
    return lso::guarded([&] { return lso::workspace_bytes(mats, n, params); }, uint64_t{0});
}

lso_status lso_orthogonalize(const lso_matrix* mats, size_t n, const lso_ns_params* params, void* workspace,
                             uint64_t workspace_bytes, void* stream)
{
    return lso::guarded([&] { return lso::run(mats, n, params, workspace, workspace_bytes, stream); }, LSO_E_NOMEM);
}

uint64_t lso_muon_workspace_bytes(const lso_muon_block* blocks, size_t n, const lso_ns_params* params)
{
    return lso::guarded([&] { return lso::workspace_bytes(blocks, n, params); }, uint64_t{0});
}

lso_status lso_muon_step(const lso_muon_block* blocks, size_t n, const lso_ns_params* params, void* workspace,
                         uint64_t workspace_bytes, void* stream)
{
    return lso::guarded([&] { return lso::run(blocks, n, params, workspace, workspace_bytes, stream); }, LSO_E_NOMEM);
}

}  // extern "C"
