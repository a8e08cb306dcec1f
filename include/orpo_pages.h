/*
 * orpo_pages.h — C ABI of beam states in shared pages, for one GB300 GPU (sm_103a).
 *
 * orpo_beam_reorder (orpo_decode.h) moves whole states when beams follow their parents.  Beams of one prompt share
 * nearly all of their past, so states kept in pages of a few positions need no more than new page numbers, and a copy of
 * at most one page per beam:
 *
 *   orpo_pages_advance   page tables follow the beams' parents (fork), and the next positions are made writable: a free page
 *                        where there is none, a copy of a page that another row holds too (copy on write)
 *   orpo_pages_copy      carries out the copies in a pool of pages
 *   orpo_pages_release   sequences that ended let go of their pages
 *   orpo_pages_compact   pages in use move to the lowest numbers
 *
 * The mlx-bun documentation pages leave generation out; the definitions below are all there is to follow.
 *
 * Data, all of it the caller's, on the device:
 *   pool   contiguous bytes [outer, pages, rows, page, unit_bytes] of any element type: e.g. outer = 2 * layers, rows = heads,
 *          page = positions per page, unit_bytes = head size * element size.  Any number of pools may share one table.
 *   table  int32 [batch * beams, columns], rows ld_table >= columns apart: position t of row r is position t % page of page
 *          table[r, t / page]; -1: no page.  Fill it with -1 at the start.
 *   refs   int32 [pages]: how many table entries hold the page; 0: the page is free.  Zero it at the start.
 *   length int32 [batch]: positions in use of an entry's rows.
 *   moves  int32 [max_moves, 3]: (from page, to page, positions), n_moves[0] of them.
 * The entry points keep refs equal to the number of table entries per page, and rely on it.  Page numbers never leave
 * [0, pages) and are checked before they are used, whatever the buffers hold.
 *
 * Conventions are those of orpo_head.h: caller-owned buffers and workspace, no allocation, asynchronous and stream-ordered
 * calls, ORPO_ERR_* return codes before any launch, ORPO_STATUS_* bits OR-ed into the device word `status`, capturable
 * in a CUDA graph.  Results do not depend on run-to-run scheduling.  All of these buffers: 4-byte aligned; workspace: 16.
 * Limits: batch >= 0, 1 <= beams <= ORPO_MAX_BEAMS, batch * beams <= 2^20, 0 <= columns, 1 <= pages <= 2^24,
 * 1 <= page <= 2^16, columns * page < 2^31, batch * beams * columns < 2^31.
 */
#ifndef ORPO_PAGES_H
#define ORPO_PAGES_H

#include "orpo_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of workspace for orpo_pages_advance with these `most` (largest number of positions asked for per call) and for
 * orpo_pages_compact, on a table of table_rows = batch * beams rows; never more than
 * 16 * pages + 64 * table_rows * (most / page + 2) + 4096.  0 for sizes out of range.
 */
size_t orpo_pages_workspace_bytes(int64_t table_rows, int64_t pages, int64_t page, int64_t most);

/*
 * One decode step of the tables, in two parts.
 * Fork (parent not NULL; int32, rows ld_parent >= beams apart), as if all rows were read before any is written:
 *   table[b, k, c] <- table[b, parent[b, k], c]   for c < ceil(length[b] / page);  refs follow.
 * Reserve: positions length[b] .. length[b] + m - 1 (m = more[b], or `most` where more is NULL; 0 <= m <= most) of every
 * row become writable.  As if the table's rows were taken in order, and in each the columns of those positions in order:
 *   no page: the lowest free page;
 *   a page that another table entry holds too (refs > 1 at its turn): the lowest free page, the entry lets go of the old one,
 *     and where positions before length[b] lie in it, (old, new, length[b] % page) is appended to moves;
 *   a page of its own: kept.
 * Free pages are those with refs = 0 after the fork.  Follow with orpo_pages_copy on every pool before the positions are
 * written.  n_moves is always set; max_moves >= batch * beams.
 * Device errors: ORPO_STATUS_PARENT (a parent outside [0, beams), more[b] outside [0, most], or positions outside [0, columns *
 * page]; that entry is left as it is), ORPO_STATUS_PAGE (a table entry outside [-1, pages); it moves with its row and is
 * otherwise left alone), ORPO_STATUS_FULL (fewer free pages than needed: the reserve part changes nothing, n_moves = 0;
 * make room and call again with parent = NULL).
 * Limits beyond those above: 0 <= most < 2^31, batch * beams * (ceil((most - 1) / page) + 1) <= 2^30.
 */
int orpo_pages_advance(int32_t* table, int64_t ld_table, int64_t columns, int32_t* refs, int64_t pages, int64_t page,
                       const int32_t* parent, int64_t ld_parent, const int32_t* length, const int32_t* more, int64_t most,
                       int64_t batch, int beams, int32_t* moves, int64_t max_moves, int32_t* n_moves, void* workspace,
                       size_t ws_bytes, int32_t* status, void* stream);

/*
 * pool[o, to, r, t, :] <- pool[o, from, r, t, :] for every move (from, to, positions), o, r and t < positions.
 * Moves run in any order: no page may be the target of one and named by another.  orpo_pages_advance and
 * orpo_pages_compact give such lists.
 * Device errors: ORPO_STATUS_PAGE (a page outside [0, pages), positions outside [0, page], from = to; that move is left out; an
 * n_moves outside [0, max_moves]: nothing moves).
 * Limits: outer, rows, unit_bytes, max_moves >= 0, max_moves < 2^31, the pool's size in bytes below 2^62,
 * page * unit_bytes < 2^31, max_moves * outer * rows * ceil(page * unit_bytes / 128) < 2^62.
 */
int orpo_pages_copy(void* pool, int64_t outer, int64_t pages, int64_t rows, int64_t page, int64_t unit_bytes,
                    const int32_t* moves, int64_t max_moves, const int32_t* n_moves, int32_t* status, void* stream);

/*
 * The rows of every entry with ended[b] != 0 (uint8 [batch]; NULL: all entries) let go of their pages: all of their table
 * entries become -1 and refs follow.  Rows without pages stay as they are.
 * Device errors: ORPO_STATUS_PAGE (a table entry outside [-1, pages), or a page whose refs are 0 already; the table entry
 * becomes -1 all the same).
 */
int orpo_pages_release(int32_t* table, int64_t ld_table, int64_t columns, int32_t* refs, int64_t pages,
                       const uint8_t* ended, int64_t batch, int beams, int32_t* status, void* stream);

/*
 * With n pages in use (refs > 0), live[0] <- n, and the pages in use that lie at n or above move to the free ones below n, the
 * i-th lowest to the i-th lowest: moves holds (page, free page, `page` positions) in that order, new_table and new_refs
 * are table and refs after the moves.  Follow with orpo_pages_copy on every pool; then pages n .. pages-1 hold nothing.
 * new_table and new_refs may be table and refs; otherwise they must not overlap them.  new_table: rows ld_new >=
 * columns apart.  max_moves >= pages / 2.
 * Device errors: ORPO_STATUS_PAGE (a table entry outside [-1, pages), or a page in the table that refs call free; copied
 * as it is).
 */
int orpo_pages_compact(const int32_t* table, int64_t ld_table, int64_t columns, int64_t table_rows, const int32_t* refs,
                       int64_t pages, int64_t page, int32_t* new_table, int64_t ld_new, int32_t* new_refs, int32_t* live,
                       int32_t* moves, int64_t max_moves, int32_t* n_moves, void* workspace, size_t ws_bytes,
                       int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ORPO_PAGES_H */
