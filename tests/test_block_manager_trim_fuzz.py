"""Differential fuzz of the host block manager with trims: a drafted step's pattern (a run of appends, then a trim) between
admissions with and without the prefix cache, forks, keying, frees and moves between two pools, id for id against the
model with a trim of its own.  What the cache gives out must hold the tokens that its key says: tokens are followed block by
block as a step would write them."""
import numpy as np
import pytest

from oracle.block_manager_ref import BlockManagerModel, NoBlocks


class Model(BlockManagerModel):
    def trim_seq(self, seq_id, num_tokens):
        blocks, n = self.seqs[seq_id]
        if not 0 <= num_tokens <= n:
            raise ValueError("bad length")
        keep = -(-num_tokens // self.block_size)
        while len(blocks) > keep:
            b = blocks.pop()
            self.ref[b] -= 1
            if self.ref[b] == 0:
                self._release(b)
        self.seqs[seq_id] = (blocks, num_tokens)

    def append_slot(self, seq_id):
        blocks, n = self.seqs[seq_id]
        if n % self.block_size and self.ref[blocks[-1]] == 1 and blocks[-1] in self.key:
            key = self.key.pop(blocks[-1])[0]     # written into: it no longer holds what its key says
            if self.index.get(key) == blocks[-1]:
                del self.index[key]
        return super().append_slot(seq_id)


@pytest.fixture(scope="module")
def binding():
    from paged_kv_cache_237_gb300 import binding
    return binding


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("bs", [4, 16])
def test_trims_between_all_other_operations_match_the_model(binding, seed, bs):
    rng = np.random.default_rng(1000 * bs + seed)
    sizes = {"dev": 1500 // bs, "host": 1500 // bs}
    lib = {k: binding.BlockManager(n, bs) for k, n in sizes.items()}
    mod = {k: Model(n, bs) for k, n in sizes.items()}
    holds = {k: {} for k in sizes}                # pool -> slot -> the token written there
    prompts = [rng.integers(0, 9, size=int(rng.integers(bs, 5 * bs))).tolist() for _ in range(4)]
    where, tokens, salt, nxt = {}, {}, {}, 0

    def both(call, fails):
        """The same call on library and model: the same result, or the same failure."""
        try:
            want = call(mod)
        except (NoBlocks, ValueError) as e:
            with pytest.raises(binding.PAError) as err:
                call(lib)
            assert err.value.code == (binding.PA_ERR_NO_BLOCKS if isinstance(e, NoBlocks) else fails)
            return None
        got = call(lib)
        if isinstance(want, list):
            got = [tuple(x) for x in got.tolist()]
        assert got == want
        return True if want is None else want

    def write(pool, seq, first):
        table = mod[pool].block_table(seq)
        for u in range(first, len(tokens[seq])):
            holds[pool][table[u // bs] * bs + u % bs] = tokens[seq][u]

    def pick(pool=None):
        live = [s for s, w in where.items() if pool is None or w == pool]
        return int(rng.choice(live)) if live else None

    for _ in range(1500):
        r, dev = rng.random(), pick("dev")
        if r < 0.14:
            p = int(rng.integers(0, 4))
            toks = prompts[p][:int(rng.integers(1, len(prompts[p]) + 1))] + rng.integers(0, 9, int(rng.integers(0, bs))).tolist()
            hit = both(lambda m: m["dev"].add_seq_cached(nxt, toks, p % 2), 0)
            if hit is not None:
                where[nxt], tokens[nxt], salt[nxt] = "dev", list(toks), p % 2
                table = mod["dev"].block_table(nxt)
                hit = 0 if hit is True else hit
                assert [holds["dev"][table[u // bs] * bs + u % bs] for u in range(hit)] == toks[:hit]
                write("dev", nxt, hit)
            nxt += 1
        elif r < 0.20:
            n = int(rng.integers(0, 4 * bs))
            if both(lambda m: m["dev"].add_seq(nxt, n), 0):
                where[nxt], tokens[nxt], salt[nxt] = "dev", rng.integers(0, 9, n).tolist(), 0
                write("dev", nxt, 0)
            nxt += 1
        elif r < 0.28 and dev is not None:
            both(lambda m: m["dev"].fork(dev, nxt), 0)
            where[nxt], tokens[nxt], salt[nxt] = "dev", list(tokens[dev]), salt[dev]
            nxt += 1
        elif r < 0.62 and where:                                       # a drafted step, or a part of one
            seq = pick()
            pool, drafted = where[seq], int(rng.integers(0, 2 * bs))
            before = len(tokens[seq])
            for _ in range(drafted):
                got = both(lambda m: tuple(m[pool].append_slot(seq)), 0)
                if got is None:
                    break
                slot, src, dst = got
                if src >= 0:
                    for o in range(bs):
                        if src * bs + o in holds[pool]:
                            holds[pool][dst * bs + o] = holds[pool][src * bs + o]
                tokens[seq].append(int(rng.integers(0, 9)))
                holds[pool][slot] = tokens[seq][-1]
            keep = int(rng.integers(before, len(tokens[seq]) + 1)) if rng.random() < 0.8 else \
                int(rng.integers(0, len(tokens[seq]) + 1))             # now and then back into the context
            both(lambda m: m[pool].trim_seq(seq, keep), 0)
            del tokens[seq][keep:]
        elif r < 0.65 and where:
            seq = pick()
            with pytest.raises(binding.PAError):
                lib[where[seq]].trim_seq(seq, len(tokens[seq]) + 1)
        elif r < 0.73 and dev is not None:
            both(lambda m: m["dev"].register_blocks(dev, tokens[dev], salt[dev]), 0)
        elif r < 0.82 and where:
            seq = pick()
            src, dst = where[seq], "host" if where[seq] == "dev" else "dev"
            pairs = both(lambda m: m[src].move_seq(m[dst], seq), binding.PA_ERR_REFCOUNT)
            if pairs is not None:
                for a, b in [] if pairs is True else pairs:
                    for o in range(bs):
                        if a * bs + o in holds[src]:
                            holds[dst][b * bs + o] = holds[src][a * bs + o]
                where[seq] = dst
        elif where:
            seq = pick()
            both(lambda m: m[where[seq]].free_seq(seq), 0)
            del where[seq], tokens[seq], salt[seq]
        for k in lib:
            assert lib[k].num_free() == mod[k].num_free() and lib[k].num_cached() == mod[k].num_cached()
        if where:
            seq = pick()
            pool = where[seq]
            table = lib[pool].block_table(seq)
            assert table == mod[pool].block_table(seq) and lib[pool].num_tokens(seq) == len(tokens[seq])
            assert [holds[pool][table[u // bs] * bs + u % bs] for u in range(len(tokens[seq]))] == tokens[seq]
    for k, n in sizes.items():
        assert [lib[k].refcount(b) for b in range(n)] == [mod[k].refcount(b) for b in range(n)]
